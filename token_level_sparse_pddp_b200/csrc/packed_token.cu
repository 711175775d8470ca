// Packed attention of few query rows (bf16, head_dim 64 or 128): the token items
// of a plan, up to 16 rows (tokens x heads of a group) against a range of keys.
//
// Memory-bound: 2 d elements are read per key and used by at most 16 rows, so
// what counts is bytes in flight, not the matrix rate; the 16 rows are exactly
// one warp-level MMA's (m16n8k16), which needs no TMEM and no hand-over between
// warps. One CTA of four warps per (item, key/value head), two CTAs per SM. Each
// warp streams its own blocks of 16 keys (every fourth block of the range)
// through a ring of three stages of 16-byte cp.async copies, with its own running
// maximum, sum and output in registers and no barrier between warps until the
// four partial outputs are joined through shared memory at the end.
// The reference maximum of a row is raised only when a score passes it by more
// than 8 (log2), so most blocks need no shuffles. Rows behind the range are
// filled with zeros; V of keys that only part of the rows see is checked for
// values that are not finite (0 x inf is NaN): those are taken out and added to
// the rows that do see them at the end.
#include "packed.h"
#include "tc_ptx.cuh"

namespace tlsp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 16;  // keys of a block
constexpr int kStages = 3;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
  static constexpr uint32_t rows = kKeys * D * 2;         // one operand of a block
  static constexpr uint32_t warp = kStages * 2 * rows;    // a warp's ring
  static constexpr uint32_t bytes = kWarps * warp;
  // after the loop: O [warp][16][D] fp32, m and l [warp][16]
  static constexpr uint32_t stat = kWarps * 16 * D * 4;
  static_assert(stat + kWarps * 32 * 4 <= bytes, "join fits into the rings");
};

struct TokenParams {
  PackedArgs a;
  float scale_log2;
  bool after;  // launched behind the tile items
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    packed_token_kernel(const __grid_constant__ TokenParams p) {
  using S = Smem<D>;
  constexpr int kChunks = D / 8;                 // 16-byte pieces of a row
  constexpr int kPer = kKeys * kChunks / 32;     // pieces a lane copies per operand
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_odd;  // own keys diag + 1 + bit whose V holds a value that is not finite
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.x % p.a.kv_heads;
  const PackedItem it = p.a.tokens[blockIdx.x / p.a.kv_heads];
  const int group = p.a.group;
  let_next_start();
  if (!item_ok(p.a, it, kTokenRows / group)) {
    if (threadIdx.x == 0) record_status(p.a.status, TLSP_ERR_DEVICE_ASSERT);
    if (p.after) wait_for_previous();
    return;
  }
  if (threadIdx.x == 0) s_odd = 0;
  __syncthreads();
  const bool pre = it.pre_n > 0;  // an item has prefix keys or own keys
  const int n = pre ? it.pre_n : min(it.kv_n, max(0, it.diag + it.nt));
  const tlsp_rows& KR = pre ? p.a.Kp : p.a.K;
  const tlsp_rows& VR = pre ? p.a.Vp : p.a.V;
  const int64_t row0 = pre ? it.pre0 : it.kv0;
  const __nv_bfloat16* K =
      static_cast<const __nv_bfloat16*>(KR.ptr) + row0 * KR.row_stride + hk * KR.head_stride;
  const __nv_bfloat16* V =
      static_cast<const __nv_bfloat16*>(VR.ptr) + row0 * VR.row_stride + hk * VR.head_stride;
  const int blocks = (n + kKeys - 1) / kKeys;
  const int mine = blocks > warp ? (blocks - warp + kWarps - 1) / kWarps : 0;

  const uint32_t ring = ptx::smem_u32(smem) + warp * S::warp;
  const int cp_chunk = lane % kChunks, cp_row = lane / kChunks;
  auto issue = [&](int b) {  // this warp's block b into its slot
    if (b < mine) {
      const int key0 = (warp + b * kWarps) * kKeys;
      const uint32_t at = ring + (b % kStages) * 2 * S::rows;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int r = cp_row + e * (32 / kChunks);
        const uint32_t dst = at + r * (D * 2) + ((cp_chunk ^ (r & 7)) * 16);
        const bool in = key0 + r < n;
        const int64_t key = in ? key0 + r : 0;
        ptx::cp_async16(dst, K + key * KR.row_stride + cp_chunk * 8, in ? 16 : 0);
        ptx::cp_async16(dst + S::rows, V + key * VR.row_stride + cp_chunk * 8, in ? 16 : 0);
      }
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int b = 0; b < kStages - 1; ++b) issue(b);

  // Q fragments: rows lane / 4 and + 8, channels 16 k + 2 (lane % 4) and + 8
  const int ra = lane >> 2, rb = ra + 8, rows = it.nt * group;
  uint32_t q[D / 16][4];
  {
    const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(p.a.Q.ptr);
    auto at = [&](int r) {
      return Q + (int64_t)(it.q0 + r / group) * p.a.Q.row_stride +
             (int64_t)(hk * group + r % group) * p.a.Q.head_stride + 2 * (lane & 3);
    };
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      q[k][0] = ra < rows ? *reinterpret_cast<const uint32_t*>(at(ra) + 16 * k) : 0u;
      q[k][1] = rb < rows ? *reinterpret_cast<const uint32_t*>(at(rb) + 16 * k) : 0u;
      q[k][2] = ra < rows ? *reinterpret_cast<const uint32_t*>(at(ra) + 16 * k + 8) : 0u;
      q[k][3] = rb < rows ? *reinterpret_cast<const uint32_t*>(at(rb) + 16 * k + 8) : 0u;
    }
  }
  // keys each row sees: the first seen (spare rows: all)
  auto seen_of = [&](int r) {
    return pre || r >= rows ? n : min(n, max(0, it.diag + r / group + 1));
  };
  const int seen_a = seen_of(ra), seen_b = seen_of(rb);
  const int every = pre ? n : min(n, max(0, it.diag + 1));  // keys that all rows see

  float o[D / 8][4];
#pragma unroll
  for (int c = 0; c < D / 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
  float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;

  for (int b = 0; b < mine; ++b) {
    const int key0 = (warp + b * kWarps) * kKeys;
    const uint32_t sk = ring + (b % kStages) * 2 * S::rows, sv = sk + S::rows;
    ptx::cp_async_wait_group<kStages - 2>();
    if (key0 + kKeys > every && every < n) {
      // each lane looks through the pieces it copied
#pragma unroll 1
      for (int e = 0; e < kPer; ++e) {
        const int r = cp_row + e * (32 / kChunks), key = key0 + r;
        if (key < every || key >= n) continue;
        const uint32_t at = sv + r * (D * 2) + ((cp_chunk ^ (r & 7)) * 16);
        uint4 w = ptx::ld_shared_v4(at);
        const uint32_t x = odd_halves(w.x), y = odd_halves(w.y), z = odd_halves(w.z),
                       u = odd_halves(w.w);
        if (x | y | z | u) {
          ptx::st_shared_v4(at, w.x & ~x, w.y & ~y, w.z & ~z, w.w & ~u);
          atomicOr(&s_odd, 1u << (key - (it.diag + 1)));
        }
      }
    }
    __syncwarp();
    issue(b + kStages - 1);  // into the slot of block b - 1, which every lane is done with

    float s[2][4] = {};
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int m = lane >> 3, r = (m >> 1) * 8 + (lane & 7), c = 2 * k + (m & 1);
      uint32_t f[4];
      ptx::ldmatrix4(sk + r * (D * 2) + ((c ^ (r & 7)) * 16), f);
      ptx::mma_16816(s[0], q[k], f[0], f[1]);
      ptx::mma_16816(s[1], q[k], f[2], f[3]);
    }
    float mxa = -INFINITY, mxb = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = key0 + 8 * t + 2 * (lane & 3) + e;
        s[t][e] = key < seen_a ? s[t][e] * p.scale_log2 : -INFINITY;
        s[t][2 + e] = key < seen_b ? s[t][2 + e] * p.scale_log2 : -INFINITY;
        mxa = fmaxf(mxa, s[t][e]);
        mxb = fmaxf(mxb, s[t][2 + e]);
      }
    if (__any_sync(0xffffffffu, mxa > ma + 8.f || mxb > mb + 8.f)) {
      auto raise = [&](float& m, float mx, float& l) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float to = fmaxf(m, mx);
        const float f = m == -INFINITY ? 0.f : ptx::ex2(m - to);
        m = to;
        l *= f;
        return f;
      };
      const float fa = raise(ma, mxa, la), fb = raise(mb, mxb, lb);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        o[c][0] *= fa;
        o[c][1] *= fa;
        o[c][2] *= fb;
        o[c][3] *= fb;
      }
    }
    const float ua = ma == -INFINITY ? 0.f : ma, ub = mb == -INFINITY ? 0.f : mb;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[t][e] = ptx::ex2(s[t][e] - ua);
        s[t][2 + e] = ptx::ex2(s[t][2 + e] - ub);
        la += s[t][e];
        lb += s[t][2 + e];
      }
    // P as the A operand (bf16, like V): 16 rows x 16 keys
    const uint32_t pf[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]),
                            pack_bf16(s[1][0], s[1][1]), pack_bf16(s[1][2], s[1][3])};
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const int m = lane >> 3, r = (m & 1) * 8 + (lane & 7), ch = 2 * c + (m >> 1);
      uint32_t f[4];
      ptx::ldmatrix4_t(sv + r * (D * 2) + ((ch ^ (r & 7)) * 16), f);
      ptx::mma_16816(o[2 * c], pf, f[0], f[1]);
      ptx::mma_16816(o[2 * c + 1], pf, f[2], f[3]);
    }
  }
  ptx::cp_async_wait_all();
  la += __shfl_xor_sync(0xffffffffu, la, 1);
  la += __shfl_xor_sync(0xffffffffu, la, 2);
  lb += __shfl_xor_sync(0xffffffffu, lb, 1);
  lb += __shfl_xor_sync(0xffffffffu, lb, 2);
  __syncthreads();

  // join the warps
  float* so = reinterpret_cast<float*>(smem);
  float* sm = reinterpret_cast<float*>(smem + S::stat);
  float* sl = sm + kWarps * 16;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    *reinterpret_cast<float2*>(&so[(warp * 16 + ra) * D + 8 * c + 2 * (lane & 3)]) =
        make_float2(o[c][0], o[c][1]);
    *reinterpret_cast<float2*>(&so[(warp * 16 + rb) * D + 8 * c + 2 * (lane & 3)]) =
        make_float2(o[c][2], o[c][3]);
  }
  if ((lane & 3) == 0) {
    sm[warp * 16 + ra] = ma;
    sm[warp * 16 + rb] = mb;
    sl[warp * 16 + ra] = la;
    sl[warp * 16 + rb] = lb;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w * 16 + r]);
    const float u = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ptx::ex2(sm[w * 16 + r] - u);
      const float4 y = *reinterpret_cast<const float4*>(&so[(w * 16 + r) * D + c]);
      l = fmaf(f, sl[w * 16 + r], l);
      x.x = fmaf(f, y.x, x.x);
      x.y = fmaf(f, y.y, x.y);
      x.z = fmaf(f, y.z, x.z);
      x.w = fmaf(f, y.w, x.w);
    }
    const bool none = l == 0.f;  // no key seen
    const float inv = none ? 0.f : 1.f / l;
    float y[4] = {none ? 0.f : x.x * inv, none ? 0.f : x.y * inv, none ? 0.f : x.z * inv,
                  none ? 0.f : x.w * inv};
    const int i = r / group, h = hk * group + r % group;
    for (uint32_t bits = s_odd; bits; bits &= bits - 1) {
      const int key = it.diag + __ffs(bits);  // diag + 1 + bit
      if (key > it.diag + i) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = __bfloat162float(V[(int64_t)key * VR.row_stride + c + k]);
        if (!(fabsf(v) < INFINITY)) y[k] += v;
      }
    }
    const float lse = none ? -INFINITY : (m + log2f(l)) * kLn2;
    if (it.slot < 0) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.O.ptr) +
                           (int64_t)(it.q0 + i) * p.a.O.row_stride + h * p.a.O.head_stride + c;
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
      if (p.a.lse && c == 0) p.a.lse[(int64_t)(it.q0 + i) * p.a.heads + h] = lse;
    } else {
      const int64_t row = (int64_t)(it.slot + i) * p.a.heads + h;
      *reinterpret_cast<float4*>(p.a.part_o + row * D + c) = make_float4(y[0], y[1], y[2], y[3]);
      if (c == 0) p.a.part_lse[row] = lse;
    }
  }
  // nothing here depends on the tile items; what follows this kernel may
  if (p.after) wait_for_previous();
}

template <int D>
int launch(const PackedArgs& a, bool after, cudaStream_t st) {
  const TokenParams p{a, a.scale * 1.4426950408889634f, after};
  auto kernel = packed_token_kernel<D>;
  TLSP_TRY(ensure_smem_limit((const void*)kernel, (int)Smem<D>::bytes));
  const dim3 grid((unsigned)((int64_t)a.n_tokens * a.kv_heads));
  if (after) return launch_after(kernel, grid, kThreads, (int)Smem<D>::bytes, st, p);
  kernel<<<grid, kThreads, Smem<D>::bytes, st>>>(p);
  return check_launch();
}

}  // namespace

int packed_token(const PackedArgs& a, bool after, cudaStream_t st) {
  return a.d == 128 ? launch<128>(a, after, st) : launch<64>(a, after, st);
}

}  // namespace tlsp
