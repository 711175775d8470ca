// Packed attention of fp32 tensors, on the CUDA cores (tensor cores round the
// operands to 19 bits or fewer).
//
// One CTA per (item, key/value head): its rows (tokens x query heads of the
// group) against blocks of 64 keys, with the running maximum and sum of the
// softmax in fp32. 256 threads as 16 x 16: a thread holds RM rows x 4 keys of
// the scores and RM rows x d / 16 channels of the output; K, V, Q and P are
// staged in shared memory as fp32.
// A masked key's V is never multiplied: rows behind the key range are stored as
// zeros, and blocks that only part of the rows see skip masked products.
#include "packed.h"

namespace tlsp {
namespace {

constexpr int kBN = 64;
constexpr int kThreads = 256;

template <int D, int BM>
constexpr int smem_floats() {
  return BM * (D + 4) + 2 * kBN * (D + 4) + BM * (kBN + 4);
}

template <int D, int BM>
__global__ void __launch_bounds__(kThreads)
    packed_simt_kernel(const __grid_constant__ PackedArgs p, const PackedItem* items) {
  constexpr int RM = BM / 16, DV = D / 16, LD = D + 4, LP = kBN + 4;
  extern __shared__ __align__(16) float sm[];
  float* sQ = sm;
  float* sK = sQ + BM * LD;
  float* sV = sK + kBN * LD;
  float* sP = sV + kBN * LD;
  const PackedItem it = items[blockIdx.x / p.kv_heads];
  const int hk = blockIdx.x % p.kv_heads;
  if (!item_ok(p, it, BM / p.group)) {
    if (threadIdx.x == 0) record_status(p.status, TLSP_ERR_DEVICE_ASSERT);
    return;
  }
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int rows = it.nt * p.group;
  const float scale = p.scale * 1.4426950408889634f;

  // Q rows r = token * group + head of the group
  const float* Q = static_cast<const float*>(p.Q.ptr);
  for (int e = threadIdx.x; e < BM * (D / 8); e += kThreads) {
    const int r = e / (D / 8), c = e % (D / 8) * 8;
    float x[8] = {};
    if (r < rows)
      load8(Q + (it.q0 + r / p.group) * p.Q.row_stride +
                (int64_t)(hk * p.group + r % p.group) * p.Q.head_stride + c,
            x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sQ[r * LD + c + i] = x[i];
  }

  float m[RM], l[RM], acc[RM][DV];
#pragma unroll
  for (int a = 0; a < RM; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
#pragma unroll
    for (int i = 0; i < DV; ++i) acc[a][i] = 0.f;
  }

  // own keys that any row sees
  const int own_n = min(it.kv_n, max(0, it.diag + it.nt));
  const int pre_blocks = (it.pre_n + kBN - 1) / kBN, own_blocks = (own_n + kBN - 1) / kBN;
  for (int blk = 0; blk < pre_blocks + own_blocks; ++blk) {
    const bool pre = blk < pre_blocks;
    const int k0 = (pre ? blk : blk - pre_blocks) * kBN;
    const int n = min(kBN, (pre ? it.pre_n : own_n) - k0);
    const tlsp_rows& KR = pre ? p.Kp : p.K;
    const tlsp_rows& VR = pre ? p.Vp : p.V;
    const int64_t row0 = (int64_t)(pre ? it.pre0 : it.kv0) + k0;
    const float* K = static_cast<const float*>(KR.ptr) + row0 * KR.row_stride + hk * KR.head_stride;
    const float* V = static_cast<const float*>(VR.ptr) + row0 * VR.row_stride + hk * VR.head_stride;
    __syncthreads();
    for (int e = threadIdx.x; e < kBN * (D / 8); e += kThreads) {
      const int r = e / (D / 8), c = e % (D / 8) * 8;
      float x[8] = {}, y[8] = {};
      if (r < n) {
        load8(K + r * KR.row_stride + c, x);
        load8(V + r * VR.row_stride + c, y);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sK[r * LD + c + i] = x[i];
        sV[r * LD + c + i] = y[i];
      }
    }
    __syncthreads();

    float s[RM][4] = {};
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
      float4 kk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<float4*>(&sK[(tx + 16 * j) * LD + k]);
#pragma unroll
      for (int a = 0; a < RM; ++a) {
        const float4 q = *reinterpret_cast<float4*>(&sQ[(ty * RM + a) * LD + k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[a][j] = fmaf(q.x, kk[j].x, s[a][j]);
          s[a][j] = fmaf(q.y, kk[j].y, s[a][j]);
          s[a][j] = fmaf(q.z, kk[j].z, s[a][j]);
          s[a][j] = fmaf(q.w, kk[j].w, s[a][j]);
        }
      }
    }
    // keys of this block that row a sees: the first seen[a]
    int seen[RM];
    bool partial = false;
#pragma unroll
    for (int a = 0; a < RM; ++a) {
      const int i = min((ty * RM + a) / p.group, it.nt - 1);  // spare rows follow the last token
      seen[a] = pre ? n : min(n, max(0, it.diag + i + 1 - k0));
      partial |= seen[a] < n;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[a][j] = tx + 16 * j < seen[a] ? s[a][j] * scale : -INFINITY;
        // fmaxf drops a NaN; it comes back through exp2f below
        mx = fmaxf(mx, s[a][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(m[a], mx);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      const float f = exp2f(m[a] - m_use);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = tx + 16 * j < seen[a] ? exp2f(s[a][j] - m_use) : 0.f;
        sum += e;
        sP[(ty * RM + a) * LP + tx + 16 * j] = e;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[a] = l[a] * f + sum;
      m[a] = m_new;
#pragma unroll
      for (int i2 = 0; i2 < DV; ++i2) acc[a][i2] *= f;
    }
    __syncwarp();  // a row's P comes from its own half warp
    if (!__any_sync(0xffffffffu, partial)) {
#pragma unroll 2
      for (int k = 0; k < kBN; k += 4) {
        float4 pr[RM];
#pragma unroll
        for (int a = 0; a < RM; ++a)
          pr[a] = *reinterpret_cast<float4*>(&sP[(ty * RM + a) * LP + k]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < DV; i += 4) {
            const float4 v = *reinterpret_cast<float4*>(&sV[(k + q) * LD + tx * 4 + i * 16]);
#pragma unroll
            for (int a = 0; a < RM; ++a) {
              const float w = q == 0 ? pr[a].x : q == 1 ? pr[a].y : q == 2 ? pr[a].z : pr[a].w;
              acc[a][i] = fmaf(w, v.x, acc[a][i]);
              acc[a][i + 1] = fmaf(w, v.y, acc[a][i + 1]);
              acc[a][i + 2] = fmaf(w, v.z, acc[a][i + 2]);
              acc[a][i + 3] = fmaf(w, v.w, acc[a][i + 3]);
            }
          }
      }
    } else {
      for (int k = 0; k < n; ++k)
#pragma unroll
        for (int a = 0; a < RM; ++a) {
          if (k >= seen[a]) continue;
          const float w = sP[(ty * RM + a) * LP + k];
#pragma unroll
          for (int i = 0; i < DV; ++i)
            acc[a][i] = fmaf(w, sV[k * LD + tx * 4 + (i / 4) * 64 + i % 4], acc[a][i]);
        }
    }
  }

#pragma unroll
  for (int a = 0; a < RM; ++a) {
    const int r = ty * RM + a;
    if (r >= rows) continue;
    const int i = r / p.group, h = hk * p.group + r % p.group;
    const bool none = l[a] == 0.f;  // no key seen
    const float inv = none ? 0.f : 1.f / l[a];
    const float lse = none ? -INFINITY : (m[a] + log2f(l[a])) * 0.6931471805599453f;
    if (it.slot < 0) {
      float* o = static_cast<float*>(p.O.ptr) + (it.q0 + i) * p.O.row_stride + h * p.O.head_stride;
#pragma unroll
      for (int c = 0; c < DV; ++c)
        o[tx * 4 + (c / 4) * 64 + c % 4] = none ? 0.f : acc[a][c] * inv;
      if (p.lse && tx == 0) p.lse[(int64_t)(it.q0 + i) * p.heads + h] = lse;
    } else {
      const int64_t row = (int64_t)(it.slot + i) * p.heads + h;
#pragma unroll
      for (int c = 0; c < DV; ++c)
        p.part_o[row * D + tx * 4 + (c / 4) * 64 + c % 4] = none ? 0.f : acc[a][c] * inv;
      if (tx == 0) p.part_lse[row] = lse;
    }
  }
}

template <int D, int BM>
int launch(const PackedArgs& a, const PackedItem* items, int n, cudaStream_t st) {
  if (n == 0) return TLSP_OK;
  auto kernel = packed_simt_kernel<D, BM>;
  constexpr int bytes = smem_floats<D, BM>() * (int)sizeof(float);
  TLSP_TRY(ensure_smem_limit((const void*)kernel, bytes));
  kernel<<<(unsigned)((int64_t)n * a.kv_heads), kThreads, bytes, st>>>(a, items);
  return check_launch();
}

template <int D>
int run(const PackedArgs& a, cudaStream_t st) {
  TLSP_TRY((launch<D, kSimtTileRows>(a, a.tiles, a.n_tiles, st)));
  return launch<D, kTokenRows>(a, a.tokens, a.n_tokens, st);
}

}  // namespace

int packed_simt(const PackedArgs& a, cudaStream_t st) {
  return a.d == 128 ? run<128>(a, st) : run<64>(a, st);
}

}  // namespace tlsp
