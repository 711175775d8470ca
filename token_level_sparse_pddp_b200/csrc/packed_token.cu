// Packed attention of few query rows (bf16, head_dim 64 or 128): the token items
// of a plan, up to 16 rows (tokens x heads of a group) against the keys of a few
// segments (the prefix, the keys of the tokens' sequences).
//
// Memory-bound: 2 d elements are read per key and used by at most 16 rows, so
// what counts is bytes in flight, not the matrix rate; the 16 rows are exactly
// one warp-level MMA's (m16n8k16), which needs no TMEM and no hand-over between
// warps. A cluster of 1 to 8 CTAs of four warps takes an (item, key/value head); two
// CTAs fit an SM. Each warp streams its own blocks of 16 keys (every n-th of the item)
// through a ring of three stages of 16-byte cp.async copies, with its own running
// maximum, sum and output in registers and no barrier between warps until the four
// partial outputs are joined in shared memory, and those of the cluster's CTAs
// through each other's: a batch of single tokens takes one launch (8 tokens behind
// 21758 cached keys, 4 heads of 128, 45 MB: 13.6 us on replay, of which some 4 us until
// the first keys are there and 2.5 us to join; two launches, with a kernel that merged the
// parts of independent CTAs, were 0.2 us slower, and 3 us more on the host). 64 channels:
// 10.9 us; 64 tokens of 4000 to 20000 keys 278 us = 5.6 TB/s.
// 64 tokens x 8 groups of 16 to 2000 keys: 41 us = 5.3 TB/s alone. Behind tile items
// (whose kernel lets it start at once) its CTAs take the SMs that those do not fill.
// The reference maximum of a row is raised only when a score passes it by more
// than 8 (log2), so most blocks need no shuffles. Rows behind a segment are filled
// with zeros; V of keys that only part of the rows see is checked for values that are
// not finite (0 x inf is NaN): those are taken out and noted for the rows that do see
// them, which get them at the end.
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
  // after the loop: O [warp][16][D] fp32, m and l [warp][16]; the CTA's O, m and l
  static constexpr uint32_t stat = kWarps * 16 * D * 4;
  static constexpr uint32_t sum = stat + kWarps * 32 * 4;
  static constexpr uint32_t sum_stat = sum + 16 * D * 4;
  static_assert(sum_stat + 32 * 4 <= bytes, "join fits into the rings");
};

struct TokenParams {
  PackedArgs a;
  float scale_log2;
  bool after;  // launched behind the tile items, on whose results nothing here depends
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// What a channel of a row got from values that are not finite, in a byte.
constexpr uint32_t kPlus = 1, kMinus = 2, kNan = 4;
__device__ __forceinline__ float odd_value(uint32_t flags) {
  if (flags & kNan || (flags & (kPlus | kMinus)) == (kPlus | kMinus)) return NAN;
  return flags & kPlus ? INFINITY : -INFINITY;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Shared memory at `addr` of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// (an aligned barrier: a warp whose lanes left a loop at different times is joined first)
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    packed_token_kernel(const __grid_constant__ TokenParams p) {
  using S = Smem<D>;
  constexpr int kChunks = D / 8;              // 16-byte pieces of a row
  constexpr int kPer = kKeys * kChunks / 32;  // pieces a lane copies per operand
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) uint32_t s_odd[16 * D / 4];  // flags of a row's channels, bytes
  __shared__ __align__(128) uint8_t s_q[16 * D * 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = p.a.cluster, unit = blockIdx.x / cluster;
  const uint32_t rank = cluster > 1 ? cluster_rank() : 0;
  const int hk = unit % p.a.kv_heads;
  const int group = p.a.group;
  for (int e = threadIdx.x; e < 16 * D / 16; e += kThreads)
    reinterpret_cast<uint4*>(s_odd)[e] = make_uint4(0, 0, 0, 0);
  // Before anything is read, the tables included: kernels before may write them. (What the
  // tile items' kernel waited for is done when this one starts behind it.)
  if (!p.after) wait_for_previous();
  let_next_start();
  const TokenItem it = p.a.token_items[unit / p.a.kv_heads];
  // Lane l holds segment l; its first block is the blocks before it.
  TokenSegment sg{};
  bool ok = it.nt >= 1 && it.nt <= kTokenRows / group && it.q0 >= 0 &&
            (int64_t)it.q0 + it.nt <= p.a.q_rows && it.seg0 >= 0 && it.nseg >= 0 &&
            it.nseg <= kMaxSegments && (int64_t)it.seg0 + it.nseg <= p.a.n_segments &&
            (it.slot < 0 || (int64_t)it.slot + it.nt <= p.a.part_rows);
  if (ok && lane < it.nseg) {
    sg = p.a.segments[it.seg0 + lane];
    ok = sg.k0 >= 0 && sg.n >= 0 && sg.tok0 >= 0 && sg.ntok >= 0 && sg.tok0 + sg.ntok <= it.nt &&
         (int64_t)sg.k0 + sg.n <= (sg.prefix ? p.a.prefix_len : p.a.kv_rows) &&
         sg.diag >= -0x40000000 && sg.diag <= sg.n;
  }
  ok = __all_sync(0xffffffffu, ok);  // the same for every warp of the cluster
  if (!ok) {
    if (p.after) wait_for_previous();
    if (threadIdx.x == 0) record_status(p.a.status, TLSP_ERR_DEVICE_ASSERT);
    return;
  }
  int first = (sg.n + kKeys - 1) / kKeys, blocks;
  {
    const int own = first;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, first, o);
      if (lane >= o) first += up;
    }
    blocks = __shfl_sync(0xffffffffu, first, 31);
    first -= own;
  }
  const int stride = kWarps * cluster, mine0 = (int)rank * kWarps + warp;
  const int mine = blocks > mine0 ? (blocks - mine0 + stride - 1) / stride : 0;
  // The segment that a warp is in; the fields come from the lane that holds it. A warp's
  // blocks ascend, so it changes rarely.
  struct Cursor {
    int first = 0, end = 0;  // blocks [first, end)
    int n, k0, tok0, ntok, diag;
    bool prefix;
  };
  auto move_to = [&](Cursor& c, int block) {
    if (block < c.end) return;
    const int q = 31 - __clz(__ballot_sync(0xffffffffu, sg.n > 0 && first <= block));
    c.n = __shfl_sync(0xffffffffu, sg.n, q);
    c.first = __shfl_sync(0xffffffffu, first, q);
    c.end = c.first + (c.n + kKeys - 1) / kKeys;
    c.k0 = __shfl_sync(0xffffffffu, sg.k0, q);
    c.tok0 = __shfl_sync(0xffffffffu, sg.tok0, q);
    c.ntok = __shfl_sync(0xffffffffu, sg.ntok, q);
    c.diag = __shfl_sync(0xffffffffu, sg.diag, q);
    c.prefix = __shfl_sync(0xffffffffu, sg.prefix, q) != 0;
  };

  const uint32_t ring = ptx::smem_u32(smem) + warp * S::warp;
  const int cp_chunk = lane % kChunks, cp_row = lane / kChunks;
  constexpr int kStep = 32 / kChunks;  // rows a warp copies at once
  const uint32_t cp_dst = cp_row * (D * 2);
  Cursor ahead;
  auto issue = [&](int b) {  // this warp's block b into its slot
    if (b < mine) {
      const int block = mine0 + b * stride;
      move_to(ahead, block);
      const tlsp_rows& KR = ahead.prefix ? p.a.Kp : p.a.K;
      const tlsp_rows& VR = ahead.prefix ? p.a.Vp : p.a.V;
      const int key = (block - ahead.first) * kKeys + cp_row;
      const int64_t row = (int64_t)ahead.k0 + key;
      const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(KR.ptr) + row * KR.row_stride +
                               hk * KR.head_stride + cp_chunk * 8;
      const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(VR.ptr) + row * VR.row_stride +
                               hk * VR.head_stride + cp_chunk * 8;
      const int64_t k_step = KR.row_stride * kStep, v_step = VR.row_stride * kStep;
      const uint32_t at = ring + (b % kStages) * 2 * S::rows + cp_dst;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const uint32_t dst = at + e * kStep * (D * 2) + ((cp_chunk ^ ((cp_row + e * kStep) & 7)) * 16);
        const bool in = key + e * kStep < ahead.n;
        // (rows behind the segment are not read: any valid address will do)
        ptx::cp_async16(dst, in ? K : static_cast<const __nv_bfloat16*>(p.a.Q.ptr), in ? 16 : 0);
        ptx::cp_async16(dst + S::rows, in ? V : static_cast<const __nv_bfloat16*>(p.a.Q.ptr),
                        in ? 16 : 0);
        K += k_step;
        V += v_step;
      }
    }
    ptx::cp_async_commit();
  };

  // Q: 16 rows in shared memory (zeros behind the last), from where each warp takes its
  // fragments: rows lane / 4 and + 8, channels 16 k + 2 (lane % 4) and + 8
  const int ra = lane >> 2, rb = ra + 8, rows = it.nt * group;
  const int ia = ra / group, ib = rb / group;  // their tokens
  for (int e = threadIdx.x; e < 16 * kChunks; e += kThreads) {
    const int r = e / kChunks, c = e % kChunks, i = r / group;
    const bool in = r < rows;
    ptx::cp_async16(ptx::smem_u32(s_q) + r * (D * 2) + ((c ^ (r & 7)) * 16),
                    static_cast<const __nv_bfloat16*>(p.a.Q.ptr) +
                        (in ? (int64_t)(it.q0 + i) * p.a.Q.row_stride +
                                  (int64_t)(hk * group + r - i * group) * p.a.Q.head_stride + c * 8
                            : 0),
                    in ? 16 : 0);
  }
  ptx::cp_async_commit();
  Cursor here;
  uint32_t q[D / 16][4];

  float o[D / 8][4];
#pragma unroll
  for (int c = 0; c < D / 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
  float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;

  // (from kStages - 1 blocks before the first, so that there is one copy of the code
  // that issues loads: a cold start fetches every instruction)
#pragma unroll 1
  for (int b = 1 - kStages; b < mine; ++b) {
    if (b < 0) {
      issue(b + kStages - 1);
      if (b == -1) {  // Q, the oldest group, and the cleared flags
        ptx::cp_async_wait_group<kStages - 1>();
        __syncthreads();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int m = lane >> 3, r = (m & 1) * 8 + (lane & 7), c = 2 * k + (m >> 1);
          ptx::ldmatrix4(ptx::smem_u32(s_q) + r * (D * 2) + ((c ^ (r & 7)) * 16), q[k]);
        }
      }
      continue;
    }
    const int block = mine0 + b * stride;
    move_to(here, block);
    const int n = here.n, key0 = (block - here.first) * kKeys;
    // keys of the segment that a token sees: the first ones (spare rows: all)
    auto seen_of = [&](int i) {
      if (here.prefix || i >= it.nt) return n;
      return i < here.tok0 || i >= here.tok0 + here.ntok
                 ? 0
                 : max(0, min(n, here.diag + i - here.tok0 + 1));
    };
    const int seen_a = seen_of(ia), seen_b = seen_of(ib);
    // that all rows see
    const int every = here.prefix ? n : here.ntok < it.nt ? 0 : max(0, min(n, here.diag + 1));
    const uint32_t sk = ring + (b % kStages) * 2 * S::rows, sv = sk + S::rows;
    ptx::cp_async_wait_group<kStages - 2>();
    if (key0 + kKeys > every && every < n) {
      // each lane looks through the pieces it copied
#pragma unroll 1
      for (int e = 0; e < kPer; ++e) {
        const int r = cp_row + e * (32 / kChunks), key = key0 + r;
        if (key < every || key >= n) continue;
        const uint32_t at = sv + r * (D * 2) + ((cp_chunk ^ (r & 7)) * 16);
        const uint4 w = ptx::ld_shared_v4(at);
        const uint32_t x = odd_halves(w.x), y = odd_halves(w.y), z = odd_halves(w.z),
                       u = odd_halves(w.w);
        if (!(x | y | z | u)) continue;
        ptx::st_shared_v4(at, w.x & ~x, w.y & ~y, w.z & ~z, w.w & ~u);
        const uint32_t half[4] = {w.x & x, w.y & y, w.z & z, w.w & u};
        uint32_t flags[2] = {0, 0};  // of eight channels
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t v = half[c >> 1] >> (16 * (c & 1)) & 0xffffu;
          if ((v & 0x7f80u) == 0x7f80u)
            flags[c >> 2] |= (v & 0x7fu ? kNan : v & 0x8000u ? kMinus : kPlus) << (8 * (c & 3));
        }
        for (int row = 0; row < rows; ++row)
          if (key < seen_of(row / group)) {
            atomicOr(&s_odd[row * (D / 4) + cp_chunk * 2], flags[0]);
            atomicOr(&s_odd[row * (D / 4) + cp_chunk * 2 + 1], flags[1]);
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
  // parts of a row: O, maximum and sum from `get`(part), joined
  struct Joined {
    float4 o;
    float m, l;
  };
  auto join = [](int parts, auto get) {
    Joined j{make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
#pragma unroll 4
    for (int x = 0; x < parts; ++x) {
      const Joined y = get(x);
      const float m = fmaxf(j.m, y.m), u = m == -INFINITY ? 0.f : m;
      const float f = ptx::ex2(j.m - u), g = ptx::ex2(y.m - u);
      j.m = m;
      j.l = fmaf(g, y.l, j.l * f);
      j.o.x = fmaf(g, y.o.x, j.o.x * f);
      j.o.y = fmaf(g, y.o.y, j.o.y * f);
      j.o.z = fmaf(g, y.o.z, j.o.z * f);
      j.o.w = fmaf(g, y.o.w, j.o.w * f);
    }
    return j;
  };
  auto of_warp = [&](int r, int c, int x) {
    return Joined{*reinterpret_cast<const float4*>(&so[(x * 16 + r) * D + c]), sm[x * 16 + r],
                  sl[x * 16 + r]};
  };
  auto finish = [&](int r, int c, const Joined& j, uint32_t flags) {
    const bool none = j.l == 0.f;  // no key seen
    const float inv = none ? 0.f : 1.f / j.l;
    float y[4] = {none ? 0.f : j.o.x * inv, none ? 0.f : j.o.y * inv, none ? 0.f : j.o.z * inv,
                  none ? 0.f : j.o.w * inv};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (flags >> (8 * k) & 0xffu) y[k] += odd_value(flags >> (8 * k) & 0xffu);
    const int i = r / group, h = hk * group + r % group;
    const float lse = none ? -INFINITY : (j.m + log2f(j.l)) * kLn2;
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
  };
  if (cluster == 1) {
    for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      finish(r, c, join(kWarps, [&](int x) { return of_warp(r, c, x); }), s_odd[e]);
    }
  } else {
    // this CTA's rows, then a share of the elements over all CTAs of the cluster
    float* to = reinterpret_cast<float*>(smem + S::sum);
    float* stat = reinterpret_cast<float*>(smem + S::sum_stat);
    for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      const Joined j = join(kWarps, [&](int x) { return of_warp(r, c, x); });
      *reinterpret_cast<float4*>(&to[r * D + c]) = j.o;
      if (c == 0) {
        stat[r] = j.m;
        stat[16 + r] = j.l;
      }
    }
    cluster_sync();
    const uint32_t a_o = ptx::smem_u32(to), a_stat = ptx::smem_u32(stat), a_odd = ptx::smem_u32(s_odd);
    for (int e = (int)rank * kThreads + threadIdx.x; e < rows * (D / 4); e += kThreads * cluster) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      uint32_t flags = 0;
      const Joined j = join(cluster, [&](int x) {
        flags |= ld_cluster(map_rank(a_odd + e * 4, x));
        return Joined{ld_cluster4(map_rank(a_o + (r * D + c) * 4, x)),
                      __uint_as_float(ld_cluster(map_rank(a_stat + r * 4, x))),
                      __uint_as_float(ld_cluster(map_rank(a_stat + (16 + r) * 4, x)))};
      });
      finish(r, c, j, flags);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
  // What follows this kernel may depend on the tile items: it ends after them.
  if (p.after && unit == (int)gridDim.x / cluster - 1) wait_for_previous();
}

template <int D>
int launch(const PackedArgs& a, bool after, cudaStream_t st) {
  const TokenParams p{a, a.scale * 1.4426950408889634f, after};
  auto kernel = packed_token_kernel<D>;
  TLSP_TRY(ensure_smem_limit((const void*)kernel, (int)Smem<D>::bytes));
  const dim3 grid((unsigned)((int64_t)a.n_tokens * a.kv_heads * a.cluster));
  return launch_dependent(kernel, grid, kThreads, (int)Smem<D>::bytes, a.cluster, st, p);
}

}  // namespace

int packed_token(const PackedArgs& a, bool after, cudaStream_t st) {
  return a.d == 128 ? launch<128>(a, after, st) : launch<64>(a, after, st);
}

}  // namespace tlsp
