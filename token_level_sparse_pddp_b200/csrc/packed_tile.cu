// Packed attention on the sm_100a tensor cores (bf16, head_dim 64 or 128): the
// tile items of a plan.
//
// One CTA per (item, key/value head). The rows of a query tile are (token, head
// of the group) pairs, so the query heads that share a key/value head share its
// K and V tiles; an item has one or two query tiles of up to 128 rows, and both
// take each chunk of 128 keys (prefix keys, then own keys) from the same shared
// memory: each key tile is read once for 256 rows.
// Warp roles (640 threads, one CTA per SM):
//   warps 0-7, 8-15 softmax and epilogue of query tile 0, 1: two threads share a row
//                   (= TMEM lane), one for keys 0-63 of each chunk, one for 64-127:
//                   four warps on each sub-partition, which keeps its special-
//                   function unit busy through each other's waits (two: 70%);
//   warp 16         lane 0 loads Q, K and V with TMA box loads (128-byte swizzle;
//                   three K and two V slots);
//   warps 17, 18    issue the tcgen05.mma instructions, Q K^T and P V (17 allocates
//                   TMEM). Each stays converged and elects one lane to issue, so
//                   that descriptors live in uniform registers (issuing from a
//                   divergent branch took 57 cycles per MMA, nearly the 64 that the
//                   MMA takes), and one's waits do not hold up the other;
//   warp 19         guards V: in the last chunk of a key range the rows behind it
//                   are zeroed, and in chunks that only part of the rows see,
//                   values that are not finite are taken out (a masked key has
//                   weight 0, and 0 x inf is NaN) and noted; the epilogue adds
//                   them to the rows that do see them.
// Per chunk and tile: S = Q K^T (fp32 in TMEM), P = 2^(S scale - m) as bf16 in
// TMEM, O += P V with A = P from TMEM. TMEM columns: one S buffer [0, 128) that
// both tiles share, P0, P1 [128, 256), O0, O1 [256, 256 + 2 d). A row's thread
// takes its whole row of S into registers at once, so the buffer is free for the
// other tile's Q K^T after some 0.2 K cycles of the softmax, and
// each tile's next scores are there when its softmax has finished. (With S of
// each tile in a buffer of its own and P written over it, a chunk of a tile went
// through softmax, P V and Q K^T one after the other: 3.5 K cycles.)
// The reference m of a row is raised (and O rescaled in TMEM) only when a chunk's
// maximum passes it by more than 8 (log2). P is rounded to bf16 (2^-8 relative,
// the type the tensor cores take); sums and O stay fp32.
// Every wait is bounded (1 s); on expiry the kernel records TLSP_ERR_TIMEOUT,
// drains its own copies and MMAs, frees TMEM and returns.
#include <algorithm>

#include "packed.h"
#include "tc_ptx.cuh"

namespace tlsp {
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 640;
constexpr int kLoadWarp = 16, kQkWarp = 17, kPvWarp = 18, kGuardWarp = 19;
constexpr int kKSlots = 3, kVSlots = 2;
constexpr uint32_t kHalfBytes = kTile * 128;  // 128 rows of 64 channels
constexpr uint32_t kTmCols = 512;
constexpr uint32_t kTmP = 128, kTmO = 256;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
  static constexpr uint32_t tile = kTile * D * 2;
  static constexpr uint32_t q = 0;
  static constexpr uint32_t k = 2 * tile;
  static constexpr uint32_t v = (2 + kKSlots) * tile;
  // 128 rows x 256 bytes of output per query tile: over its Q where that is as large
  static constexpr uint32_t stage_bytes = kTile * 256;
  static constexpr uint32_t stage = D == 128 ? q : (2 + kKSlots + kVSlots) * tile;
  static constexpr uint32_t bar = (2 + kKSlots + kVSlots) * tile + (D == 128 ? 0 : 2 * stage_bytes);
  static constexpr uint32_t bytes = bar + 512 + 1024;  // + slack to align the base
};

struct Bars {
  uint64_t q_full;
  uint64_t k_full[kKSlots], k_empty[kKSlots];
  uint64_t v_full[kVSlots], v_ready[kVSlots], v_empty[kVSlots];
  uint64_t s_full[2], s_free, p_full[2], pv_done[2], drain[2];
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

// Bit 15 and bit 31 tell which bf16 halves of a word are not finite (exponent all
// ones: adding one to it carries into the sign's place).
__device__ __forceinline__ uint32_t exp_carry(uint32_t w) {
  return (w & 0x7f807f80u) + 0x00800080u;
}
// All bits of those halves.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// Barrier of `threads` threads; true if `vote` was, in any of them.
__device__ __forceinline__ bool bar_or(int id, int threads, bool vote) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)vote), "r"(id), "r"(threads)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
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
      ptx::mbar_init(&bars.p_full[s], 8);  // warps
      ptx::mbar_init(&bars.pv_done[s], 1);
    }
    ptx::mbar_init(&bars.s_free, 8);
    ptx::mbar_init(&bars.drain[0], 1);
    ptx::mbar_init(&bars.drain[1], 1);
    bars.abort = 0;
    for (int i = 0; i < 8; ++i) bars.odd[i] = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kQkWarp) {
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
  } else if (warp == kQkWarp || warp == kPvWarp) {
    // ------------------------------------------------------------ MMA issuers
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && ptx::mbar_spin(bar, parity & 1, abort_flag, kWaitNs);
    };
    if (warp == kQkWarp && n_chunks > 0) {
      constexpr uint32_t id_qk = ptx::idesc_bf16(kTile, kTile, false);
      wait(&bars.q_full, 0);
      int scores = 0;  // Q K^T issued so far
      for (int j = 0; j < n_chunks; ++j) {
        wait(&bars.k_full[j % kKSlots], j / kKSlots);
#pragma unroll
        for (int s = 0; s < 2; ++s) {  // S = Q_s K_j^T, once the S before has been read
          if (j >= (s == 0 ? n0 : n1)) continue;
          if (scores > 0) wait(&bars.s_free, scores - 1);
          ++scores;
          if (!__all_sync(0xffffffffu, ok)) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint64_t qd = ptx::sw128_desc(base + S::q + s * S::tile, 16, 1024);
            const uint64_t kd = ptx::sw128_desc(base + S::k + (j % kKSlots) * S::tile, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32u;
              ptx::mma_ss(tmem, qd + (off >> 4), kd + (off >> 4), id_qk, kk > 0 ? 1u : 0u);
            }
            ptx::tc_commit(&bars.s_full[s]);
            if (s == 1 || j >= n1) ptx::tc_commit(&bars.k_empty[j % kKSlots]);  // its last use
          }
          __syncwarp();
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
    }
    if (warp == kPvWarp) {
      constexpr uint32_t id_pv = ptx::idesc_bf16(kTile, D, true);
      for (int j = 0; j < n_chunks; ++j) {
        wait(&bars.v_ready[j % kVSlots], j / kVSlots);
#pragma unroll
        for (int s = 0; s < 2; ++s) {  // O_s += P_s V_j
          if (j >= (s == 0 ? n0 : n1)) continue;
          wait(&bars.p_full[s], j);
          if (!__all_sync(0xffffffffu, ok)) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint64_t vd =
                ptx::sw128_desc(base + S::v + (j % kVSlots) * S::tile, kHalfBytes, 1024);
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              ptx::mma_ts(tmem + kTmO + s * D, tmem + kTmP + s * 64 + kk * 8,
                          vd + kk * (2048 >> 4), id_pv, (j > 0 || kk > 0) ? 1u : 0u);
            ptx::tc_commit(&bars.pv_done[s]);
            if (s == 1 || j >= n1) ptx::tc_commit(&bars.v_empty[j % kVSlots]);
          }
          __syncwarp();
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
    }
    // all issued MMAs must land before TMEM is released, even after an abort
    uint64_t* drain = &bars.drain[warp - kQkWarp];
    __syncwarp();
    if (ptx::elect_one()) {
      if (!ok) fail(bars, p.a.status);
      ptx::tc_commit(drain);
    }
    __syncwarp();
    ptx::mbar_wait(drain, 0, nullptr, kWaitNs);
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
        const uint32_t v = base + S::v + vs * S::tile;
        for (int h = 0; h < kHalves; ++h) {
          const uint32_t rows = v + h * kHalfBytes;  // 8 x 16 bytes a row
          const int first = every * 8 + lane, end = some * 8;
          // eight pieces at a time; the usual answer is that all are finite
          for (int u = first; u < end; u += 256) {
            uint4 w[8];
            uint32_t odd = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              w[e] = u + 32 * e < end ? ptx::ld_shared_v4(rows + (u + 32 * e) * 16)
                                      : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              odd |= exp_carry(w[e].x) | exp_carry(w[e].y) | exp_carry(w[e].z) | exp_carry(w[e].w);
            if (!(odd & 0x80008000u)) continue;
#pragma unroll 1
            for (int x = u; x < min(end, u + 256); x += 32) {
              uint4 y = ptx::ld_shared_v4(rows + x * 16);
              const uint32_t a = odd_halves(y.x), b = odd_halves(y.y), c = odd_halves(y.z),
                             d = odd_halves(y.w);
              if (!(a | b | c | d)) continue;
              ptx::st_shared_v4(rows + x * 16, y.x & ~a, y.y & ~b, y.z & ~c, y.w & ~d);
              const int bit = (j - pre_chunks) * kTile + x / 8 - (it.diag + 1);
              atomicOr(&bars.odd[bit >> 5], 1u << (bit & 31));
            }
          }
          for (int u = end + lane; u < kTile * 8; u += 32) ptx::st_shared_v4(rows + u * 16, 0, 0, 0, 0);
        }
        ptx::fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.v_ready[vs]);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int s = warp >> 3;           // query tile
    const int half = (warp >> 2) & 1;  // keys 64 half .. + 63 of each chunk
    const int r = tid & 127;           // row
    const int pair = 1 + s * 4 + (warp & 3);  // barrier of the two warps of 32 rows
    const int i = r / group + s * p.tile_tokens, h = hk * group + r % group;
    const int nt = s == 0 ? nt0 : it.nt, n = s == 0 ? n0 : n1;
    const bool real = i < nt && r < p.tile_tokens * group;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = tl + 64 * half, p_col = tl + kTmP + s * 64;
    constexpr int kCols = D / 2;  // of O, for this thread
    const uint32_t o_col = tl + kTmO + s * D + half * kCols;
    float m_run = -INFINITY, l_run = 0.f;
    // own keys that this row sees (spare rows: all), and that every row of the warp sees
    const int own_seen = real ? max(0, min(it.kv_n, it.diag + i + 1)) : 0x7fffffff;
    const int own_whole = __reduce_min_sync(0xffffffffu, own_seen);
    // After a failure the warp runs on without waiting (its partner waits for it at
    // the pair's barriers), on whatever TMEM holds; nothing is written out then.
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      if (ok && !ptx::mbar_spin(bar, parity & 1, abort_flag, kWaitNs)) {
        ok = false;
        fail(bars, p.a.status);
      }
      __syncwarp();
      ptx::tc_fence_after();
    };
    for (int j = 0; j < n; ++j) {
      // this thread's keys of the chunk: the row sees the first `seen`
      const int at = (j < pre_chunks ? j : j - pre_chunks) * kTile + 64 * half;
      const bool whole = at + 64 <= (j < pre_chunks ? it.pre_n : own_whole);
      wait(&bars.s_full[s], j);
      uint32_t c[2][32];  // the row's scores
      ptx::tmem_ld32(s_col, c[0]);
      ptx::tmem_ld32(s_col + 32, c[1]);
      ptx::tmem_ld_wait(c[0]);
      ptx::reg_barrier(c[1]);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.s_free);
      if (!whole) {  // masked scores become -inf under either sign of the scale
        const uint32_t off = p.scale_log2 < 0.f ? 0x7f800000u : 0xff800000u;
        const int seen = (j < pre_chunks ? it.pre_n : own_seen) - at;
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e >= seen) c[e / 32][e % 32] = off;
      }
      // their maximum (fmaxf drops a NaN; it comes back through ex2)
      float mx;
      if (p.scale_log2 >= 0.f) {
        float t[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          t[b] = __uint_as_float(c[b][0]);
#pragma unroll
          for (int e = 1; e + 1 < 32; e += 2)
            t[b] = ptx::max3(t[b], __uint_as_float(c[b][e]), __uint_as_float(c[b][e + 1]));
        }
        mx = fmaxf(ptx::max3(t[0], t[1], __uint_as_float(c[0][31])), __uint_as_float(c[1][31]));
      } else {
        mx = INFINITY;
#pragma unroll
        for (int e = 0; e < 64; ++e) mx = fminf(mx, __uint_as_float(c[e / 32][e % 32]));
      }
      mx *= p.scale_log2;
      // Raise the reference? The rows' two warps go together (TMEM accesses are
      // warp-collective); rows that need no raise move by less than 8. Spare rows
      // do not vote.
      if (bar_or(pair, 64, real && mx > m_run + 8.f)) {
        // once P's columns are free the two threads of a row swap their maxima there
        if (j > 0) wait(&bars.pv_done[s], j - 1);
        ptx::tmem_st1(p_col + 32 * half, __float_as_uint(mx));
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        bar_sync(pair, 64);
        ptx::tc_fence_after();
        const float m_new =
            ptx::max3(m_run, mx, __uint_as_float(ptx::tmem_ld1(p_col + 32 * (1 - half))));
        if (j > 0) {  // O *= 2^(m_run - m_new)
          const float f = m_run == -INFINITY ? 0.f : ptx::ex2(m_run - m_new);
#pragma unroll 1
          for (int q = 0; q < kCols / 16; ++q) {
            uint32_t o[16];
            ptx::tmem_ld16(o_col + q * 16, o);
            ptx::tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            ptx::tmem_st16(o_col + q * 16, o);
          }
          l_run *= f;
        }
        m_run = m_new;
        ptx::tc_fence_before();
        bar_sync(pair, 64);  // both have read before P is written
        ptx::tc_fence_after();
      }
      const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
      const uint64_t sc2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
      const uint64_t nm2 = ptx::f2_pack(neg_m, neg_m);
      uint64_t sum2[2] = {0ull, 0ull};
      uint32_t pk[32];  // P, pairs of bf16
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const uint64_t x =
            ptx::f2_fma(ptx::f2_pack(__uint_as_float(c[e / 16][2 * (e % 16)]),
                                     __uint_as_float(c[e / 16][2 * (e % 16) + 1])),
                        sc2, nm2);
        float x0, x1;
        ptx::f2_unpack(x, x0, x1);
        const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
        sum2[e & 1] = ptx::f2_add(sum2[e & 1], ptx::f2_pack(p0, p1));
        pk[e] = pack_bf16(p0, p1);
      }
      float a0, a1, a2, a3;
      ptx::f2_unpack(sum2[0], a0, a1);
      ptx::f2_unpack(sum2[1], a2, a3);
      l_run += (a0 + a1) + (a2 + a3);
      if (j > 0) wait(&bars.pv_done[s], j - 1);  // the P before has been taken
      ptx::tmem_st32(p_col + 32 * half, pk);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.p_full[s]);
    }
    if (n > 0) wait(&bars.pv_done[s], n - 1);
    // The query tile's shared memory (its Q K^T are done) joins the two halves of the
    // row's sum, then stages the rows: a warp writes whole rows (each thread its own
    // row, 16 bytes at a time, took 8 to 19 us an item, with the rows' distance).
    float* sums = reinterpret_cast<float*>(smem + S::stage + s * S::stage_bytes);
    if (n > 0) sums[half * kTile + r] = l_run;
    ok = __all_sync(0xffffffffu, ok);
    ok = !bar_or(9 + s, 256, !ok);
    if (ok) {
      const float l = n > 0 ? sums[r] + sums[kTile + r] : 0.f;
      const bool none = l == 0.f;  // no key seen
      const float inv = none ? 0.f : 1.f / l;
      const bool part = it.slot >= 0;
      if (real && half == 0) {
        const float lse = none ? -INFINITY : (m_run + log2f(l)) * kLn2;
        if (part)
          p.a.part_lse[(int64_t)(it.slot + i) * p.a.heads + h] = lse;
        else if (p.a.lse)
          p.a.lse[(int64_t)(it.q0 + i) * p.a.heads + h] = lse;
      }
      bar_sync(9 + s, 256);  // the sums have been read
      uint32_t any_odd = 0;
      for (int w = 0; w < 8; ++w) any_odd |= bars.odd[w];
      const uint32_t stage = base + S::stage + s * S::stage_bytes;
      const int rows = (nt - s * p.tile_tokens) * group;  // real rows of the tile
#pragma unroll 1
      for (int q = 0; q < kCols / 32; ++q) {
        const int c0 = half * kCols + q * 32;  // first channel
        uint32_t o[32];
        if (n > 0) {
          ptx::tmem_ld32(o_col + q * 32, o);
          ptx::tmem_ld_wait(o);
        }
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = none ? 0.f : __uint_as_float(o[e]) * inv;
        if (any_odd && real) {
          for (int w = 0; w < 8; ++w)
            for (uint32_t bits = bars.odd[w]; bits; bits &= bits - 1) {
              const int key = it.diag + 1 + 32 * w + __ffs(bits) - 1;
              if (key > it.diag + i) continue;
              const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.a.V.ptr) +
                                       (int64_t)(it.kv0 + key) * p.a.V.row_stride +
                                       hk * p.a.V.head_stride + c0;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float y = __bfloat162float(v[e]);
                if (!(fabsf(y) < INFINITY)) x[e] += y;
              }
            }
        }
        if (part) {  // 32 channels of each half at a time: rows of 256 bytes
#pragma unroll
          for (int c = 0; c < 8; ++c)
            ptx::st_shared_v4(stage + r * 256 + (((half * 8 + c) ^ (r & 7)) * 16),
                              __float_as_uint(x[4 * c]), __float_as_uint(x[4 * c + 1]),
                              __float_as_uint(x[4 * c + 2]), __float_as_uint(x[4 * c + 3]));
          bar_sync(9 + s, 256);
          for (int e = tid & 255; e < rows * 16; e += 256) {
            const int rr = e >> 4, c = e & 15;
            const uint4 v = ptx::ld_shared_v4(stage + rr * 256 + ((c ^ (rr & 7)) * 16));
            float* to = p.a.part_o +
                        ((int64_t)(it.slot + rr / group + s * p.tile_tokens) * p.a.heads +
                         hk * group + rr % group) * D;
            *reinterpret_cast<uint4*>(to + (c >> 3) * kCols + q * 32 + (c & 7) * 4) = v;
          }
          bar_sync(9 + s, 256);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            ptx::st_shared_v4(stage + r * (D * 2) + (((c0 / 8 + c) ^ (r & 7)) * 16),
                              pack_bf16(x[8 * c], x[8 * c + 1]), pack_bf16(x[8 * c + 2], x[8 * c + 3]),
                              pack_bf16(x[8 * c + 4], x[8 * c + 5]), pack_bf16(x[8 * c + 6], x[8 * c + 7]));
        }
      }
      if (!part) {
        bar_sync(9 + s, 256);
        for (int e = tid & 255; e < rows * (D / 8); e += 256) {
          const int rr = e / (D / 8), c = e % (D / 8);
          const uint4 v = ptx::ld_shared_v4(stage + rr * (D * 2) + ((c ^ (rr & 7)) * 16));
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.a.O.ptr) +
                              (int64_t)(it.q0 + rr / group + s * p.tile_tokens) * p.a.O.row_stride +
                              (int64_t)(hk * group + rr % group) * p.a.O.head_stride;
          *reinterpret_cast<uint4*>(to + c * 8) = v;
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
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
