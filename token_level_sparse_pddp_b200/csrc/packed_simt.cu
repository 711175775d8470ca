// Packed attention of fp32 tensors, on the CUDA cores (tensor cores round the
// operands to 19 bits or fewer).
//
// One CTA per (item, key/value head): its rows (tokens x query heads of the group)
// against blocks of 64 keys, with the running maximum and sum of the softmax.
// 16 threads share RM rows: each holds RM x 4 scores and RM x d / 16 channels of O.
// Bound: fp32 FMA (and, below it, shared-memory reads: 12 wavefronts of a warp's
// operands per 64 FMAs). Scores and products are accumulated two at a time
// (fma .f32x2), which leaves issue slots for the reads. K and V have one buffer each,
// filled by 16-byte cp.async while the other is used: V(j) comes in under Q K(j)^T,
// K(j + 1) under P V(j).
// Measured, six ragged sequences (1850 tokens, 2989 keys, 8 / 2 heads, d = 64):
// 65.8 us = 23 TFLOP/s, with the merge; 8 x 1024 queries and keys without mask 35 TFLOP/s
// (packed FMAs alone reach 64 in a loop on registers; shared-memory wavefronts are 74%
// busy, the FMA pipe 57%; 64-row items and 8 rows per thread measured within 3% of this).
// 64 single tokens of 12 / 4 heads of 128 behind 4000 to 20000 keys each: 1160 us = 2.7
// TB/s, as 3 of an item's 16 rows are filled (22 TFLOP/s with the others counted).
// A masked key has weight 0, and 0 x inf is NaN: rows behind the key range are stored
// as zeros, and a block that only part of the rows see is searched for values that are
// not finite; with one, masked products are skipped.
#include "packed.h"
#include "tc_ptx.cuh"

namespace tlsp {
namespace {

constexpr int kBN = 64;

template <int D, int BM, int RM>
struct Config {
  static constexpr int threads = 16 * BM / RM;
  static constexpr int ld = D + 4;   // row strides that spread over the banks
  static constexpr int lp = kBN + 4;
  static constexpr int bytes = (BM * ld + 2 * kBN * ld + BM * lp) * (int)sizeof(float);
};

template <int D, int BM, int RM>
__global__ void __launch_bounds__(Config<D, BM, RM>::threads)
    packed_simt_kernel(const __grid_constant__ PackedArgs p, const PackedItem* items, bool after) {
  using C = Config<D, BM, RM>;
  constexpr int DV = D / 16, LD = C::ld, LP = C::lp, kThreads = C::threads;
  extern __shared__ __align__(16) float sm[];
  float* sQ = sm;
  float* sK = sQ + BM * LD;
  float* sV = sK + kBN * LD;
  float* sP = sV + kBN * LD;
  // Before anything is read, the table included: kernels before may write it. (What the
  // tile items' kernel waited for is done when the token items' starts.)
  if (!after) wait_for_previous();
  let_next_start();
  const PackedItem it = items[blockIdx.x / p.kv_heads];
  const int hk = blockIdx.x % p.kv_heads;
  if (!item_ok(p, it, BM / p.group)) {
    if (after) wait_for_previous();
    if (threadIdx.x == 0) record_status(p.status, TLSP_ERR_DEVICE_ASSERT);
    return;
  }
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int rows = it.nt * p.group;
  const float scale = p.scale * 1.4426950408889634f;

  // own keys that any row sees
  const int own_n = min(it.kv_n, max(0, it.diag + it.nt));
  const int pre_blocks = (it.pre_n + kBN - 1) / kBN;
  const int blocks = pre_blocks + (own_n + kBN - 1) / kBN;
  // first key of a block, and how many of its keys count
  auto keys_of = [&](int blk, int& k0) {
    const bool pre = blk < pre_blocks;
    k0 = (pre ? blk : blk - pre_blocks) * kBN;
    return min(kBN, (pre ? it.pre_n : own_n) - k0);
  };
  // Block `blk` of K or V into shared memory; rows behind the range as zeros.
  auto fetch = [&](const tlsp_rows& pre_rows, const tlsp_rows& own_rows, int blk, float* to) {
    if (blk < blocks) {
      int k0;
      const int n = keys_of(blk, k0);
      const bool pre = blk < pre_blocks;
      const tlsp_rows& R = pre ? pre_rows : own_rows;
      const float* from = static_cast<const float*>(R.ptr) +
                          ((int64_t)(pre ? it.pre0 : it.kv0) + k0) * R.row_stride + hk * R.head_stride;
      const uint32_t dst = ptx::smem_u32(to);
#pragma unroll 4
      for (int e = threadIdx.x; e < kBN * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        ptx::cp_async16(dst + (r * LD + c) * 4, from + (r < n ? r : 0) * R.row_stride + c,
                        r < n ? 16 : 0);
      }
    }
    ptx::cp_async_commit();
  };
  fetch(p.Kp, p.K, 0, sK);
  fetch(p.Vp, p.V, 0, sV);

  // Q rows r = token * group + head of the group
  for (int e = threadIdx.x; e < BM * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
      x = *reinterpret_cast<const float4*>(
          static_cast<const float*>(p.Q.ptr) + (it.q0 + r / p.group) * p.Q.row_stride +
          (int64_t)(hk * p.group + r % p.group) * p.Q.head_stride + c);
    *reinterpret_cast<float4*>(&sQ[r * LD + c]) = x;
  }
  int own_seen[RM];  // own keys each row sees (spare rows follow the last token)
#pragma unroll
  for (int a = 0; a < RM; ++a)
    own_seen[a] = max(0, min(own_n, it.diag + 1 + min((ty * RM + a) / p.group, it.nt - 1)));

  float m[RM], l[RM];
  uint64_t acc[RM][DV / 2];  // channel pairs
#pragma unroll
  for (int a = 0; a < RM; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
#pragma unroll
    for (int i = 0; i < DV / 2; ++i) acc[a][i] = 0ull;
  }

  for (int blk = 0; blk < blocks; ++blk) {
    int k0;
    const int n = keys_of(blk, k0);
    const bool pre = blk < pre_blocks;
    ptx::cp_async_wait_group<1>();  // K(blk)
    __syncthreads();
    uint64_t s2[RM][4];
#pragma unroll
    for (int a = 0; a < RM; ++a)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[a][j] = 0ull;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
      ulonglong2 kk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<ulonglong2*>(&sK[(tx + 16 * j) * LD + k]);
#pragma unroll
      for (int a = 0; a < RM; ++a) {
        const ulonglong2 q = *reinterpret_cast<ulonglong2*>(&sQ[(ty * RM + a) * LD + k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s2[a][j] = ptx::f2_fma(q.x, kk[j].x, s2[a][j]);
          s2[a][j] = ptx::f2_fma(q.y, kk[j].y, s2[a][j]);
        }
      }
    }
    __syncthreads();  // K is free
    fetch(p.Kp, p.K, blk + 1, sK);

    // keys of this block that row a sees: the first seen[a]
    int seen[RM];
    float s[RM][4], mx[RM], sum[RM];
#pragma unroll
    for (int a = 0; a < RM; ++a) {
      seen[a] = pre ? n : min(n, max(0, own_seen[a] - k0));
      mx[a] = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float lo, hi;
        ptx::f2_unpack(s2[a][j], lo, hi);
        s[a][j] = tx + 16 * j < seen[a] ? (lo + hi) * scale : -INFINITY;
        mx[a] = fmaxf(mx[a], s[a][j]);  // drops a NaN; it comes back through exp2f below
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int a = 0; a < RM; ++a) mx[a] = fmaxf(mx[a], __shfl_xor_sync(0xffffffffu, mx[a], o));
#pragma unroll
    for (int a = 0; a < RM; ++a) {
      const float m_new = fmaxf(m[a], mx[a]), m_use = m_new == -INFINITY ? 0.f : m_new;
      const float f = exp2f(m[a] - m_use);
      m[a] = m_new;
      l[a] *= f;
      const uint64_t f2 = ptx::f2_pack(f, f);
#pragma unroll
      for (int i = 0; i < DV / 2; ++i) acc[a][i] = ptx::f2_fma(acc[a][i], f2, 0ull);
      sum[a] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = tx + 16 * j < seen[a] ? exp2f(s[a][j] - m_use) : 0.f;
        sum[a] += e;
        sP[(ty * RM + a) * LP + tx + 16 * j] = e;
      }
      l[a] += sum[a];  // this thread's keys; joined at the end
    }
    ptx::cp_async_wait_group<1>();  // V(blk)
    __syncthreads();                // of all threads; and P of a row's 16
    bool odd = false;
    // (the first token of the item sees the fewest keys)
    if (!pre && it.diag + 1 - k0 < n) {
      for (int e = threadIdx.x; e < kBN * (D / 4); e += kThreads) {
        const float4 v = *reinterpret_cast<float4*>(&sV[e / (D / 4) * LD + e % (D / 4) * 4]);
        odd |= !(fabsf(v.x) < INFINITY) || !(fabsf(v.y) < INFINITY) || !(fabsf(v.z) < INFINITY) ||
               !(fabsf(v.w) < INFINITY);
      }
      odd = __syncthreads_or(odd);
    }
    if (!odd) {
#pragma unroll 2
      for (int k = 0; k < kBN; k += 4) {
        float4 pr[RM];
#pragma unroll
        for (int a = 0; a < RM; ++a)
          pr[a] = *reinterpret_cast<float4*>(&sP[(ty * RM + a) * LP + k]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint64_t w2[RM];
#pragma unroll
          for (int a = 0; a < RM; ++a) {
            const float w = q == 0 ? pr[a].x : q == 1 ? pr[a].y : q == 2 ? pr[a].z : pr[a].w;
            w2[a] = ptx::f2_pack(w, w);
          }
#pragma unroll
          for (int i = 0; i < DV; i += 4) {
            const ulonglong2 v = *reinterpret_cast<ulonglong2*>(&sV[(k + q) * LD + tx * 4 + i * 16]);
#pragma unroll
            for (int a = 0; a < RM; ++a) {
              acc[a][i / 2] = ptx::f2_fma(w2[a], v.x, acc[a][i / 2]);
              acc[a][i / 2 + 1] = ptx::f2_fma(w2[a], v.y, acc[a][i / 2 + 1]);
            }
          }
        }
      }
    } else {
      for (int k = 0; k < n; ++k)
#pragma unroll
        for (int a = 0; a < RM; ++a) {
          if (k >= seen[a]) continue;
          const float w = sP[(ty * RM + a) * LP + k];
          const uint64_t w2 = ptx::f2_pack(w, w);
#pragma unroll
          for (int i = 0; i < DV; i += 4) {
            const ulonglong2 v = *reinterpret_cast<ulonglong2*>(&sV[k * LD + tx * 4 + i * 16]);
            acc[a][i / 2] = ptx::f2_fma(w2, v.x, acc[a][i / 2]);
            acc[a][i / 2 + 1] = ptx::f2_fma(w2, v.y, acc[a][i / 2 + 1]);
          }
        }
    }
    __syncthreads();  // V and P are free
    fetch(p.Vp, p.V, blk + 1, sV);
  }
  ptx::cp_async_wait_all();

#pragma unroll
  for (int a = 0; a < RM; ++a) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) l[a] += __shfl_xor_sync(0xffffffffu, l[a], o);
    const int r = ty * RM + a;
    if (r >= rows) continue;
    const int i = r / p.group, h = hk * p.group + r % p.group;
    const bool none = l[a] == 0.f;  // no key seen
    const float inv = none ? 0.f : 1.f / l[a];
    const float lse = none ? -INFINITY : (m[a] + log2f(l[a])) * 0.6931471805599453f;
    float* o;
    if (it.slot < 0) {
      o = static_cast<float*>(p.O.ptr) + (it.q0 + i) * p.O.row_stride + h * p.O.head_stride;
      if (p.lse && tx == 0) p.lse[(int64_t)(it.q0 + i) * p.heads + h] = lse;
    } else {
      const int64_t row = (int64_t)(it.slot + i) * p.heads + h;
      o = p.part_o + row * D;
      if (tx == 0) p.part_lse[row] = lse;
    }
#pragma unroll
    for (int c = 0; c < DV; c += 4) {
      float4 y;
      ptx::f2_unpack(acc[a][c / 2], y.x, y.y);
      ptx::f2_unpack(acc[a][c / 2 + 1], y.z, y.w);
      y = none ? make_float4(0.f, 0.f, 0.f, 0.f)
               : make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      *reinterpret_cast<float4*>(o + tx * 4 + c * 16) = y;
    }
  }
  // What follows this kernel may depend on the tile items: it ends after them.
  if (after && blockIdx.x == gridDim.x - 1) wait_for_previous();
}

template <int D, int BM, int RM>
int launch(const PackedArgs& a, const PackedItem* items, int n, bool after, cudaStream_t st) {
  if (n == 0) return TLSP_OK;
  using C = Config<D, BM, RM>;
  auto kernel = packed_simt_kernel<D, BM, RM>;
  TLSP_TRY(ensure_smem_limit((const void*)kernel, C::bytes));
  return launch_dependent(kernel, dim3((unsigned)((int64_t)n * a.kv_heads)), C::threads, C::bytes, 1, st, a,
                          items, after);
}

template <int D>
int run(const PackedArgs& a, cudaStream_t st) {
  if (simt_tile_rows(a.group) == 32)
    TLSP_TRY((launch<D, 32, 4>(a, a.tiles, a.n_tiles, false, st)));
  else
    TLSP_TRY((launch<D, 64, 4>(a, a.tiles, a.n_tiles, false, st)));
  return launch<D, kTokenRows, 2>(a, a.tokens, a.n_tokens, a.n_tiles > 0, st);
}

}  // namespace

int packed_simt(const PackedArgs& a, cudaStream_t st) {
  return a.d == 128 ? run<128>(a, st) : run<64>(a, st);
}

}  // namespace tlsp
