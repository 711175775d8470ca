// Packed attention on the sm_100a tensor cores (bf16, head_dim 64 or 128): the
// tile items of a plan.
//
// One CTA per (item, key/value head). The rows of a query tile are (token, head
// of the group) pairs, so the query heads that share a key/value head share its
// K and V tiles; an item has one or two query tiles of up to 128 rows, and both
// take each chunk of 128 keys (prefix keys, then own keys) from the same shared
// memory: each key tile is read once for 256 rows.
// Warp roles (384 threads, one CTA per SM):
//   warps 0-3, 4-7  softmax and epilogue of query tile 0, 1: thread t owns row t
//                   = TMEM lane t;
//   warp 8          lane 0 loads Q, K and V with TMA box loads (128-byte swizzle;
//                   three K and two V slots);
//   warp 9          allocates TMEM; lane 0 issues the tcgen05.mma instructions;
//   warp 10         guards V: in the last chunk of a key range the rows behind it
//                   are zeroed, and in chunks that only part of the rows see,
//                   values that are not finite are taken out (a masked key has
//                   weight 0, and 0 x inf is NaN) and noted; the epilogue adds
//                   them to the rows that do see them.
// Per chunk and tile: S = Q K^T (fp32 in TMEM), P = 2^(S scale - m) in one pass,
// written over S as bf16, O += P V with A = P from TMEM. The two tiles take turns:
// while one's softmax runs, the tensor cores work on the other's P V and next
// Q K^T. TMEM columns: S0, S1 [0, 256), O0, O1 [256, 256 + 2 d).
// The reference m of a row is the maximum of the first 32 scores it sees; it is
// raised (and O rescaled in TMEM) only when a chunk's sum of P exceeds 2^8, which
// any score more than 8 (in log2) above m causes. P is rounded to bf16 (2^-8
// relative, the type the tensor cores take); sums and O stay fp32.
// Every wait is bounded (1 s); on expiry the kernel records TLSP_ERR_TIMEOUT,
// drains its own copies and MMAs, frees TMEM and returns.
#include <algorithm>

#include "packed.h"
#include "tc_ptx.cuh"

namespace tlsp {
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 384;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kGuardWarp = 10;
constexpr int kKSlots = 3, kVSlots = 2;
constexpr uint32_t kHalfBytes = kTile * 128;  // 128 rows of 64 channels
constexpr uint32_t kTmCols = 512;
constexpr uint32_t kTmO = 256;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
  static constexpr uint32_t tile = kTile * D * 2;
  static constexpr uint32_t q = 0;
  static constexpr uint32_t k = 2 * tile;
  static constexpr uint32_t v = (2 + kKSlots) * tile;
  static constexpr uint32_t bar = (2 + kKSlots + kVSlots) * tile;
  static constexpr uint32_t bytes = bar + 512 + 1024;  // + slack to align the base
};

struct Bars {
  uint64_t q_full;
  uint64_t k_full[kKSlots], k_empty[kKSlots];
  uint64_t v_full[kVSlots], v_ready[kVSlots], v_empty[kVSlots];
  uint64_t s_full[2], p_full[2], o_final[2], drain;
  uint32_t tmem_base;
  int abort;
  uint32_t odd[8];  // own keys diag + 1 + bit whose V holds a value that is not finite
};
static_assert(sizeof(Bars) <= 512, "barrier block");

struct TileParams {
  PackedArgs a;
  CUtensorMap tmQ, tmK, tmV, tmKp, tmVp;
  int tile_tokens;  // of one query tile
  float scale_log2;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ void fail(Bars& b, int* status) {
  *(volatile int*)&b.abort = 1;
  record_status(status, TLSP_ERR_TIMEOUT);
}

// Both bf16 halves of a word: bits of those that are not finite.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_tile_kernel(const __grid_constant__ TileParams p) {
  using S = Smem<D>;
  constexpr int kHalves = D / 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  Bars& bars = *reinterpret_cast<Bars*>(smem + S::bar);
  volatile int* abort_flag = &bars.abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x % p.a.kv_heads;
  const PackedItem it = p.a.tiles[blockIdx.x / p.a.kv_heads];
  if (!item_ok(p.a, it, 2 * p.tile_tokens)) {
    if (tid == 0) record_status(p.a.status, TLSP_ERR_DEVICE_ASSERT);
    return;
  }
  const int group = p.a.group;
  // tokens of the two query tiles and the chunks each of them takes
  const int nt0 = min(it.nt, p.tile_tokens), nt1 = it.nt - nt0;
  const int pre_chunks = (it.pre_n + kTile - 1) / kTile;
  const int seen0 = max(0, min(it.kv_n, it.diag + nt0));
  const int seen1 = max(0, min(it.kv_n, it.diag + it.nt));
  const int n0 = pre_chunks + (seen0 + kTile - 1) / kTile;
  const int n1 = nt1 > 0 ? pre_chunks + (seen1 + kTile - 1) / kTile : 0;
  const int n_chunks = max(n0, n1);

  if (tid == 0) {
    ptx::mbar_init(&bars.q_full, 1);
    for (int s = 0; s < kKSlots; ++s) {
      ptx::mbar_init(&bars.k_full[s], 1);
      ptx::mbar_init(&bars.k_empty[s], 1);
    }
    for (int s = 0; s < kVSlots; ++s) {
      ptx::mbar_init(&bars.v_full[s], 1);
      ptx::mbar_init(&bars.v_ready[s], 1);
      ptx::mbar_init(&bars.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bars.s_full[s], 1);
      ptx::mbar_init(&bars.p_full[s], 128);
      ptx::mbar_init(&bars.o_final[s], 1);
    }
    ptx::mbar_init(&bars.drain, 1);
    bars.abort = 0;
    for (int i = 0; i < 8; ++i) bars.odd[i] = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&bars.tmem_base, kTmCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars.tmem_base;

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0 && n_chunks > 0) {
      const uint32_t q_bytes = (uint32_t)(p.tile_tokens * group) * D * 2;  // one box's rows
      ptx::mbar_arrive_expect_tx(&bars.q_full, (nt1 > 0 ? 2 : 1) * q_bytes);
      for (int s = 0; s < (nt1 > 0 ? 2 : 1); ++s)
        for (int h = 0; h < kHalves; ++h)
          ptx::tma_load_4d(base + S::q + s * S::tile + h * kHalfBytes, &p.tmQ, 64 * h, 0, hk,
                           it.q0 + s * p.tile_tokens, &bars.q_full);
      int issued_k = 0, issued_v = 0;
      bool ok = true;
      for (int j = 0; j < n_chunks; ++j) {
        const int ks = j % kKSlots, ku = j / kKSlots, vs = j % kVSlots, vu = j / kVSlots;
        const bool pre = j < pre_chunks;
        const CUtensorMap* mk = pre ? &p.tmKp : &p.tmK;
        const CUtensorMap* mv = pre ? &p.tmVp : &p.tmV;
        const int y = pre ? it.pre0 + j * kTile : it.kv0 + (j - pre_chunks) * kTile;
        if (ku > 0 && !ptx::mbar_wait(&bars.k_empty[ks], (ku - 1) & 1, abort_flag, kWaitNs)) {
          ok = false;
          break;
        }
        ptx::mbar_arrive_expect_tx(&bars.k_full[ks], S::tile);
        for (int h = 0; h < kHalves; ++h)
          ptx::tma_load_3d(base + S::k + ks * S::tile + h * kHalfBytes, mk, 64 * h, hk, y,
                           &bars.k_full[ks]);
        issued_k = j + 1;
        if (vu > 0 && !ptx::mbar_wait(&bars.v_empty[vs], (vu - 1) & 1, abort_flag, kWaitNs)) {
          ok = false;
          break;
        }
        ptx::mbar_arrive_expect_tx(&bars.v_full[vs], S::tile);
        for (int h = 0; h < kHalves; ++h)
          ptx::tma_load_3d(base + S::v + vs * S::tile + h * kHalfBytes, mv, 64 * h, hk, y,
                           &bars.v_full[vs]);
        issued_v = j + 1;
      }
      if (!ok) {
        fail(bars, p.a.status);
        // loads already issued land before the CTA's shared memory goes away
        for (int j = max(0, issued_k - kKSlots); j < issued_k; ++j)
          ptx::mbar_wait(&bars.k_full[j % kKSlots], (j / kKSlots) & 1, nullptr, kWaitNs);
        for (int j = max(0, issued_v - kVSlots); j < issued_v; ++j)
          ptx::mbar_wait(&bars.v_full[j % kVSlots], (j / kVSlots) & 1, nullptr, kWaitNs);
        ptx::mbar_wait(&bars.q_full, 0, nullptr, kWaitNs);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && n_chunks > 0) {
      constexpr uint32_t id_qk = ptx::idesc_bf16(kTile, kTile, false);
      constexpr uint32_t id_pv = ptx::idesc_bf16(kTile, D, true);
      bool ok = ptx::mbar_wait(&bars.q_full, 0, abort_flag, kWaitNs);
      auto qk = [&](int s, int j) {  // S_s = Q_s K_j^T
        const uint32_t qb = base + S::q + s * S::tile, kb = base + S::k + (j % kKSlots) * S::tile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32u;
          ptx::mma_ss(tmem + s * kTile, ptx::sw128_desc(qb + off, 16, 1024),
                      ptx::sw128_desc(kb + off, 16, 1024), id_qk, kk > 0 ? 1u : 0u);
        }
        ptx::tc_commit(&bars.s_full[s]);
      };
      auto pv = [&](int s, int j) {  // O_s += P_s V_j
        const uint32_t vb = base + S::v + (j % kVSlots) * S::tile;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          ptx::mma_ts(tmem + kTmO + s * D, tmem + s * kTile + kk * 8,
                      ptx::sw128_desc(vb + kk * 2048, kHalfBytes, 1024), id_pv,
                      (j > 0 || kk > 0) ? 1u : 0u);
      };
      auto wait_k = [&](int j) {
        ok = ok && ptx::mbar_wait(&bars.k_full[j % kKSlots], (j / kKSlots) & 1, abort_flag, kWaitNs);
        ptx::tc_fence_after();
      };
      wait_k(0);
      if (ok) {
        if (n0 > 0) qk(0, 0);
        if (n1 > 0) qk(1, 0);
        ptx::tc_commit(&bars.k_empty[0]);
      }
      for (int j = 0; j < n_chunks && ok; ++j) {
        // the last tile that takes chunk j (and j + 1) releases its slots
        ok = ptx::mbar_wait(&bars.v_ready[j % kVSlots], (j / kVSlots) & 1, abort_flag, kWaitNs);
        if (j + 1 < n_chunks) wait_k(j + 1);
        const bool last1 = j < n1;
#pragma unroll 1
        for (int s = 0; s < 2 && ok; ++s) {
          const int n = s == 0 ? n0 : n1;
          if (j >= n) continue;
          ok = ptx::mbar_wait(&bars.p_full[s], j & 1, abort_flag, kWaitNs);
          if (!ok) break;
          ptx::fence_proxy_async_smem();
          ptx::tc_fence_after();
          pv(s, j);
          if (s == 1 || !last1) ptx::tc_commit(&bars.v_empty[j % kVSlots]);
          if (j == n - 1) ptx::tc_commit(&bars.o_final[s]);
          if (j + 1 < n) {
            qk(s, j + 1);
            if (s == 1 || j + 1 >= n1) ptx::tc_commit(&bars.k_empty[(j + 1) % kKSlots]);
          }
        }
      }
      if (!ok) fail(bars, p.a.status);
      // all issued MMAs must land before TMEM is released
      ptx::tc_commit(&bars.drain);
      ptx::mbar_wait(&bars.drain, 0, nullptr, kWaitNs);  // even after an abort
    }
    __syncwarp();
  } else if (warp == kGuardWarp) {
    // ------------------------------------------------------------ V guard
    for (int j = 0; j < n_chunks; ++j) {
      const int vs = j % kVSlots;
      if (!ptx::mbar_wait(&bars.v_full[vs], (j / kVSlots) & 1, abort_flag, kWaitNs)) {
        if (lane == 0) fail(bars, p.a.status);
        break;
      }
      // chunk rows [0, every) are seen by all rows of the item, [every, some) by
      // part of them, the others by none
      int every, some;
      if (j < pre_chunks) {
        every = some = min(kTile, it.pre_n - j * kTile);
      } else {
        const int c = (j - pre_chunks) * kTile;
        some = min(kTile, seen1 - c);
        every = min(some, max(0, it.diag + 1 - c));
      }
      if (every < kTile) {
        uint8_t* v = smem + S::v + vs * S::tile;
        for (int h = 0; h < kHalves; ++h) {
          uint4* rows = reinterpret_cast<uint4*>(v + h * kHalfBytes);  // 8 x 16 bytes a row
#pragma unroll 4
          for (int u = every * 8 + lane; u < some * 8; u += 32) {
            uint4 w = rows[u];
            const uint32_t a = odd_halves(w.x), b = odd_halves(w.y), c = odd_halves(w.z),
                           d = odd_halves(w.w);
            if (a | b | c | d) {
              w.x &= ~a;
              w.y &= ~b;
              w.z &= ~c;
              w.w &= ~d;
              rows[u] = w;
              const int bit = (j - pre_chunks) * kTile + u / 8 - (it.diag + 1);
              atomicOr(&bars.odd[bit >> 5], 1u << (bit & 31));
            }
          }
          for (int u = some * 8 + lane; u < kTile * 8; u += 32) rows[u] = make_uint4(0, 0, 0, 0);
        }
        ptx::fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.v_ready[vs]);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int s = warp >> 2;  // query tile
    const int r = tid & 127;  // row
    const int i = r / group + s * p.tile_tokens, h = hk * group + r % group;
    const int nt = s == 0 ? nt0 : it.nt, n = s == 0 ? n0 : n1;
    const bool real = i < nt && r < p.tile_tokens * group;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = tl + s * kTile, o_col = tl + kTmO + s * D;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      // keys of the chunk that this row sees: the first `seen` (spare rows: all)
      int seen = kTile;
      if (real) {
        if (j < pre_chunks) {
          seen = it.pre_n - j * kTile;
        } else {
          const int c = (j - pre_chunks) * kTile;
          seen = min(it.kv_n, it.diag + i + 1) - c;
        }
        seen = min(kTile, max(0, seen));
      }
      const bool whole = __all_sync(0xffffffffu, seen == kTile);
      if (!ptx::mbar_wait(&bars.s_full[s], j & 1, abort_flag, kWaitNs)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      uint32_t pk[64];  // the chunk's P, pairs of bf16
      // P = 2^(S scale - m) of the whole chunk; returns its sum
      auto p_pass = [&](float m_ref) {
        const float neg_m = -m_ref;
        const uint64_t sc2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
        const uint64_t nm2 = ptx::f2_pack(neg_m, neg_m);
        uint64_t sum2[2] = {0ull, 0ull};
        auto block = [&](const uint32_t (&cur)[32], int b) {
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t x = ptx::f2_fma(
                  ptx::f2_pack(__uint_as_float(cur[2 * e]), __uint_as_float(cur[2 * e + 1])), sc2,
                  nm2);
              float x0, x1;
              ptx::f2_unpack(x, x0, x1);
              const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
              sum2[e & 1] = ptx::f2_add(sum2[e & 1], ptx::f2_pack(p0, p1));
              pk[16 * b + e] = pack_bf16(p0, p1);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int c0 = 32 * b + 2 * e;
              const float x0 = fmaf(__uint_as_float(cur[2 * e]), p.scale_log2, neg_m);
              const float x1 = fmaf(__uint_as_float(cur[2 * e + 1]), p.scale_log2, neg_m);
              const float p0 = c0 < seen ? ptx::ex2(x0) : 0.f;
              const float p1 = c0 + 1 < seen ? ptx::ex2(x1) : 0.f;
              sum2[e & 1] = ptx::f2_add(sum2[e & 1], ptx::f2_pack(p0, p1));
              pk[16 * b + e] = pack_bf16(p0, p1);
            }
          }
        };
        uint32_t ra[32], rb[32];
        ptx::tmem_ld32(s_col, ra);
        ptx::tmem_ld32(s_col + 32, rb);
        ptx::tmem_ld_wait(ra);
        ptx::reg_barrier(rb);
        block(ra, 0);
        ptx::tmem_ld32(s_col + 64, ra);
        block(rb, 1);
        ptx::tmem_ld32(s_col + 96, rb);
        ptx::tmem_ld_wait(ra);
        ptx::reg_barrier(rb);
        block(ra, 2);
        block(rb, 3);
        float a, b, c, d;
        ptx::f2_unpack(sum2[0], a, b);
        ptx::f2_unpack(sum2[1], c, d);
        return (a + b) + (c + d);
      };
      // maximum of the seen scores among the first `cols` (log2 units)
      auto max_pass = [&](int cols) {
        float pm[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int b = 0; b < cols / 32; ++b) {
          uint32_t c[32];
          ptx::tmem_ld32(s_col + 32 * b, c);
          ptx::tmem_ld_wait(c);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * b + e < seen)
              pm[e & 1] = fmaxf(pm[e & 1], __uint_as_float(c[e]) * p.scale_log2);
        }
        return fmaxf(pm[0], pm[1]);
      };
      if (j == 0) m_run = max_pass(32);
      float sum = p_pass(m_run == -INFINITY ? 0.f : m_run);
      // A row whose sum is too large, or that sees its first scores only now
      // (further right than the first 32, or all of them -inf so far), takes the
      // chunk's true maximum. TMEM accesses are warp-collective: the warp goes
      // together, rows that need no raise keep their reference or raise it by
      // less than 2^8. Spare rows do not vote.
      if (__any_sync(0xffffffffu,
                     real && (!(sum <= 256.f) || (m_run == -INFINITY && seen > 0)))) {
        const float m_new = fmaxf(max_pass(kTile), m_run);
        if (j > 0) {
          // S_j is complete, so the P V before it is too: O *= 2^(m_run - m_new)
          const float f = m_run == -INFINITY ? 0.f : ptx::ex2(m_run - m_new);
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            ptx::tmem_ld32(o_col + q * 32, o);
            ptx::tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            ptx::tmem_st32(o_col + q * 32, o);
          }
          l_run *= f;
        }
        m_run = m_new;
        sum = p_pass(m_run == -INFINITY ? 0.f : m_run);
      }
      l_run += sum;
      // every score has been read: P goes over the first 64 of S's columns
      ptx::tmem_st32(s_col, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
      ptx::tmem_st32(s_col + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bars.p_full[s]);
    }
    if (ok && n > 0 && !ptx::mbar_wait(&bars.o_final[s], 0, abort_flag, kWaitNs)) ok = false;
    if (!ok) {
      fail(bars, p.a.status);
    } else {
      ptx::tc_fence_after();
      const bool none = l_run == 0.f;  // no key seen
      const float inv = none ? 0.f : 1.f / l_run;
      const float lse = none ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
      const bool part = it.slot >= 0;
      const int64_t part_row = (int64_t)((part ? it.slot : 0) + i) * p.a.heads + h;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.O.ptr) +
                           (int64_t)(it.q0 + i) * p.a.O.row_stride + h * p.a.O.head_stride;
      if (real) {
        if (part)
          p.a.part_lse[part_row] = lse;
        else if (p.a.lse)
          p.a.lse[(int64_t)(it.q0 + i) * p.a.heads + h] = lse;
      }
      uint32_t any_odd = 0;
      for (int w = 0; w < 8; ++w) any_odd |= bars.odd[w];
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        if (n > 0) {
          ptx::tmem_ld32(o_col + q * 32, o);  // every lane: the load is warp-collective
          ptx::tmem_ld_wait(o);
        }
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = none ? 0.f : __uint_as_float(o[e]) * inv;
        if (!real) continue;
        if (any_odd) {
          for (int w = 0; w < 8; ++w)
            for (uint32_t bits = bars.odd[w]; bits; bits &= bits - 1) {
              const int key = it.diag + 1 + 32 * w + __ffs(bits) - 1;
              if (key > it.diag + i) continue;
              const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.a.V.ptr) +
                                       (int64_t)(it.kv0 + key) * p.a.V.row_stride +
                                       hk * p.a.V.head_stride + q * 32;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float y = __bfloat162float(v[e]);
                if (!(fabsf(y) < INFINITY)) x[e] += y;
              }
            }
        }
        if (part) {
          float4* dst = reinterpret_cast<float4*>(p.a.part_o + part_row * D + q * 32);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            dst[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(out + q * 32);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            dst[c] = make_uint4(pack_bf16(x[8 * c], x[8 * c + 1]), pack_bf16(x[8 * c + 2], x[8 * c + 3]),
                                pack_bf16(x[8 * c + 4], x[8 * c + 5]), pack_bf16(x[8 * c + 6], x[8 * c + 7]));
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmCols);
  }
}

// [rows, kv_heads, d] as (channel, head, row), boxes of 64 channels x 128 rows
int kv_map(CUtensorMap* map, const tlsp_rows& r, int64_t rows, int heads, int d) {
  if (rows == 0) return TLSP_OK;  // never loaded from
  const uint64_t dims[3] = {(uint64_t)d, (uint64_t)heads, (uint64_t)rows};
  const uint64_t strides[2] = {(uint64_t)r.head_stride, (uint64_t)r.row_stride};
  const uint32_t box[3] = {64, 1, kTile};
  return make_tmap_bf16(map, r.ptr, 3, dims, strides, box);
}

template <int D>
int launch(const PackedArgs& a, cudaStream_t st) {
  TileParams p{};
  p.a = a;
  p.tile_tokens = kTcRows / a.group;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  // Q as (channel, head of the group, key/value head, token)
  const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.group, (uint64_t)a.kv_heads, (uint64_t)a.q_rows};
  const uint64_t strides[3] = {(uint64_t)a.Q.head_stride, (uint64_t)a.Q.head_stride * a.group,
                               (uint64_t)a.Q.row_stride};
  const uint32_t box[4] = {64, (uint32_t)a.group, 1, (uint32_t)p.tile_tokens};
  TLSP_TRY(make_tmap_bf16(&p.tmQ, a.Q.ptr, 4, dims, strides, box));
  TLSP_TRY(kv_map(&p.tmK, a.K, a.kv_rows, a.kv_heads, D));
  TLSP_TRY(kv_map(&p.tmV, a.V, a.kv_rows, a.kv_heads, D));
  TLSP_TRY(kv_map(&p.tmKp, a.Kp, a.prefix_len, a.kv_heads, D));
  TLSP_TRY(kv_map(&p.tmVp, a.Vp, a.prefix_len, a.kv_heads, D));
  auto kernel = packed_tile_kernel<D>;
  TLSP_TRY(ensure_smem_limit((const void*)kernel, (int)Smem<D>::bytes));
  kernel<<<(unsigned)((int64_t)a.n_tiles * a.kv_heads), kThreads, Smem<D>::bytes, st>>>(p);
  return check_launch();
}

}  // namespace

int packed_tile(const PackedArgs& a, cudaStream_t st) {
  return a.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace tlsp
