// Packed attention on the sm_100a tensor cores (bf16, head_dim 64 or 128): the
// tile items of a plan.
//
// The rows of a query tile are (token, head of the group) pairs, so the query
// heads that share a key/value head share its K and V tiles; an item has one or
// two query tiles of up to 128 rows, and both take each chunk of 128 keys from the
// same shared memory: each key tile is read once for 256 rows. Chunks are taken from
// the last own key down to the first, then from the prefix's end to its start: what
// only part of the rows see comes first, while the item before is being finished.
//
// The grid has a block per (item, key/value head), longest first. A resident block
// that has finished takes over blocks that have not started (launch control: no
// counter in memory), so the items are handed out as SMs come free, while loads
// and Q K^T of the next item run under the softmax and epilogue of the last (a
// block per item spent 10 us on starting, filling and draining: 40% of the time of
// 24 ragged prompts).
//
// Warp roles (640 threads, one CTA per SM):
//   warps 0-7, 8-15 softmax and epilogue of query tile 0, 1: two threads share a row
//                   (= TMEM lane), one for keys 0-63 of each chunk, one for 64-127:
//                   four warps on each sub-partition, which keeps its special-
//                   function unit busy through each other's waits (two: 70%);
//   warp 16         lane 0 loads Q, K and V with TMA box loads (128-byte swizzle;
//                   two K and two V slots);
//   warps 17, 18    issue the tcgen05.mma instructions, Q K^T and P V (17 allocates
//                   TMEM). Each stays converged and elects one lane to issue, so
//                   that descriptors live in uniform registers (issuing from a
//                   divergent branch took 57 cycles per MMA, nearly the 64 that the
//                   MMA takes), and one's waits do not hold up the other;
//   warp 19         guards V: in the last chunk of a key range the rows behind it
//                   are zeroed, and in chunks that only part of the rows see,
//                   values that are not finite are taken out (a masked key has
//                   weight 0, and 0 x inf is NaN) and noted; the epilogue adds
//                   them to the rows that do see them. It also fetches the items,
//                   one ahead.
// Per chunk and tile: S = Q K^T (fp32 in TMEM), P = 2^(S scale - m) as bf16 in
// TMEM, O += P V with A = P from TMEM. TMEM columns: one S buffer [0, 128) that
// both tiles share, P0, P1 [128, 256), O0, O1 [256, 256 + 2 d). The threads take
// their rows of S into registers at once, so the buffer is free for the other
// tile's Q K^T after some 0.2 K cycles, and each tile's next scores are there when
// its softmax has finished. (With S of each tile in a buffer of its own and P
// written over it, a chunk of a tile went through softmax, P V and Q K^T one after
// the other: 3.5 K cycles for both tiles, against 2.0 K of the tensor cores' and of
// the special-function units' work.)
// The reference m of a row is raised (and O rescaled in TMEM) only when a chunk's
// maximum passes it by more than 8 (log2). P is rounded to bf16 (2^-8 relative,
// the type the tensor cores take); sums and O stay fp32.
// Bound: a chunk of both tiles takes the tensor cores 2.0 K cycles (32 MMAs of 64) and
// the special-function units 2.0 K (32768 exponentials at 16 a cycle); each is busy for
// 75% of the cycles of 16384 causal tokens of 12 heads of 128 (610 us; shared memory,
// DRAM 5%). 32760 tokens: 2.30 ms = 1.43 PFLOP/s on a cool GPU, 2.70 ms = 1.22 PFLOP/s
// back to back, where the power limit holds the clock at 1.47 GHz. An item takes 4.5 us
// besides its chunks (1.5 us each): getting it, the first maximum, the last P V, the
// way out.
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
constexpr int kSlots = 2;  // of K, and of V
constexpr uint32_t kHalfBytes = kTile * 128;   // 128 rows of 64 channels
constexpr uint32_t kTmCols = 512;
constexpr uint32_t kTmP = 128, kTmO = 256;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
  static constexpr uint32_t tile = kTile * D * 2;
  static constexpr uint32_t q = 0;
  static constexpr uint32_t k = 2 * tile;
  static constexpr uint32_t v = k + kSlots * tile;
  static constexpr uint32_t sums = v + kSlots * tile;  // fp32 [query tile][half][row]
  static constexpr uint32_t bar = sums + 4 * kTile * 4;
  static constexpr uint32_t bytes = bar + 512 + 1024;  // + slack to align the base
};

// An item as the roles see it.
struct Work {
  PackedItem it;
  int hk;      // key/value head
  int blocks;  // 0: no more items
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[kSlots], k_empty[kSlots];
  uint64_t v_full[kSlots], v_ready[kSlots], v_empty[kSlots];
  uint64_t s_full[2], s_free, p_full[2], pv_done[2], drain[2];
  uint64_t work_full[2], work_empty[2], answer_full;
  uint4 answer;
  Work work[2];
  uint32_t odd[2][8];  // own keys diag + 1 + bit whose V holds a value that is not finite
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");
constexpr int kWorkReaders = 3 + 16;  // warps that read an item: loads, MMAs, softmax

struct TileParams {
  PackedArgs a;
  CUtensorMap tmQ, tmK, tmV, tmKp, tmVp;
  int tile_tokens;  // of one query tile
  uint32_t magic;   // row / group = row magic >> 16, rows < 128
  float scale_log2;
};

// The chunks of an item: prefix chunks [0, pre), own chunks behind them. Tile 0
// takes chunks n0 - 1 .. 0, tile 1 chunks n1 - 1 .. 0 (n1 >= n0 or n1 = 0).
struct Shape {
  int nt0, nt1;      // tokens of the query tiles
  int pre;           // prefix chunks
  int seen1;         // own keys that any row sees
  int n0, n1, most;  // chunks of the tiles, and of the longer one
  __device__ __forceinline__ Shape(const PackedItem& it, int tile_tokens) {
    nt0 = min(it.nt, tile_tokens);
    nt1 = it.nt - nt0;
    pre = (it.pre_n + kTile - 1) / kTile;
    const int seen0 = max(0, min(it.kv_n, it.diag + nt0));
    seen1 = max(0, min(it.kv_n, it.diag + it.nt));
    n0 = pre + (seen0 + kTile - 1) / kTile;
    n1 = nt1 > 0 ? pre + (seen1 + kTile - 1) / kTile : 0;
    most = max(n0, n1);
  }
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

// Barrier of `threads` threads; true if `vote` was, in any of them. (These barriers count
// threads; what follows them here, TMEM accesses, asks for converged warps.)
__device__ __forceinline__ bool bar_or(int id, int threads, bool vote) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)vote), "r"(id), "r"(threads)
      : "memory");
  __syncwarp();
  return any != 0;
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
  __syncwarp();
}

// 640 threads start with 96 registers each; the 512 of the softmax need a few more
// than that, the other four warps fewer: 512 x 104 + 128 x 64 <= 640 x 96.
__device__ __forceinline__ void set_regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
}
__device__ __forceinline__ void set_regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
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
  const int group = p.a.group;

  if (tid == kGuardWarp * 32) {
    ptx::mbar_init(&bars.q_full, 1);
    ptx::mbar_init(&bars.q_empty, 1);
    for (int s = 0; s < kSlots; ++s) {
      ptx::mbar_init(&bars.k_full[s], 1);
      ptx::mbar_init(&bars.k_empty[s], 1);
      ptx::mbar_init(&bars.v_full[s], 1);
      ptx::mbar_init(&bars.v_ready[s], 1);
      ptx::mbar_init(&bars.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bars.s_full[s], 1);
      ptx::mbar_init(&bars.p_full[s], 8);  // warps
      ptx::mbar_init(&bars.pv_done[s], 1);
      ptx::mbar_init(&bars.drain[s], 1);
      ptx::mbar_init(&bars.work_full[s], 1);
      ptx::mbar_init(&bars.work_empty[s], kWorkReaders);
    }
    ptx::mbar_init(&bars.s_free, 8);
    ptx::mbar_init(&bars.answer_full, 1);
    bars.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kQkWarp) {
    ptx::tmem_alloc(&bars.tmem_base, kTmCols);
    ptx::tmem_relinquish();
  }
  if (tid == kLoadWarp * 32) {
    ptx::prefetch_tmap(&p.tmQ);
    if (p.a.kv_rows > 0) {
      ptx::prefetch_tmap(&p.tmK);
      ptx::prefetch_tmap(&p.tmV);
    }
    if (p.a.prefix_len > 0) {
      ptx::prefetch_tmap(&p.tmKp);
      ptx::prefetch_tmap(&p.tmVp);
    }
  }
  wait_for_previous();
  let_next_start();  // token items run on SMs that this kernel does not fill
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars.tmem_base;

  // Item number `k` of this block: false when there is none (or after a failure).
  auto next_work = [&](int k, Work& w) {
    if (!ptx::mbar_spin(&bars.work_full[k & 1], (k >> 1) & 1, abort_flag, kWaitNs)) {
      fail(bars, p.a.status);
      return false;
    }
    w = bars.work[k & 1];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&bars.work_empty[k & 1]);
    return w.blocks != 0;
  };

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ TMA producer
    set_regs_less();
    const uint32_t q_bytes = (uint32_t)(p.tile_tokens * group) * D * 2;  // a box's rows
    int c = 0, items = 0;  // chunks and items with any, so far
    bool ok = true;
    Work w;
    for (int k = 0; ok && next_work(k, w); ++k) {
      const Shape sh(w.it, p.tile_tokens);
      if (sh.most == 0) continue;
      if (lane == 0) {
        auto wait = [&](uint64_t* bar, int parity) {
          ok = ok && ptx::mbar_wait(bar, parity & 1, abort_flag, kWaitNs);
          return ok;
        };
        if (items == 0 || wait(&bars.q_empty, items - 1)) {
          ptx::mbar_arrive_expect_tx(&bars.q_full, (sh.nt1 > 0 ? 2 : 1) * q_bytes);
          for (int s = 0; s < (sh.nt1 > 0 ? 2 : 1); ++s)
            for (int h = 0; h < kHalves; ++h)
              ptx::tma_load_4d(base + S::q + s * S::tile + h * kHalfBytes, &p.tmQ, 64 * h, 0, w.hk,
                               w.it.q0 + s * p.tile_tokens, &bars.q_full);
          ++items;
        }
        for (int j = sh.most - 1; j >= 0 && ok; --j) {
          const int slot = c % kSlots, use = c / kSlots;
          const bool pre = j < sh.pre;
          const CUtensorMap* mk = pre ? &p.tmKp : &p.tmK;
          const CUtensorMap* mv = pre ? &p.tmVp : &p.tmV;
          const int y = pre ? w.it.pre0 + j * kTile : w.it.kv0 + (j - sh.pre) * kTile;
          if (use > 0 && !wait(&bars.k_empty[slot], use - 1)) break;
          ptx::mbar_arrive_expect_tx(&bars.k_full[slot], S::tile);
          for (int h = 0; h < kHalves; ++h)
            ptx::tma_load_3d(base + S::k + slot * S::tile + h * kHalfBytes, mk, 64 * h, w.hk, y,
                             &bars.k_full[slot]);
          if (use > 0 && !wait(&bars.v_empty[slot], use - 1)) {
            // the K load just issued lands before the shared memory goes away
            ptx::mbar_wait(&bars.k_full[slot], use & 1, nullptr, kWaitNs);
            break;
          }
          ptx::mbar_arrive_expect_tx(&bars.v_full[slot], S::tile);
          for (int h = 0; h < kHalves; ++h)
            ptx::tma_load_3d(base + S::v + slot * S::tile + h * kHalfBytes, mv, 64 * h, w.hk, y,
                             &bars.v_full[slot]);
          ++c;
        }
        if (!ok) {
          fail(bars, p.a.status);
          for (int x = max(0, c - kSlots); x < c; ++x) {
            ptx::mbar_wait(&bars.k_full[x % kSlots], (x / kSlots) & 1, nullptr, kWaitNs);
            ptx::mbar_wait(&bars.v_full[x % kSlots], (x / kSlots) & 1, nullptr, kWaitNs);
          }
          if (items > 0) ptx::mbar_wait(&bars.q_full, (items - 1) & 1, nullptr, kWaitNs);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
  } else if (warp == kQkWarp || warp == kPvWarp) {
    // ------------------------------------------------------------ MMA issuers
    set_regs_less();
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {
      ok = ok && ptx::mbar_spin(bar, parity & 1, abort_flag, kWaitNs);
    };
    Work w;
    int c = 0;  // chunks so far
    if (warp == kQkWarp) {
      constexpr uint32_t id_qk = ptx::idesc_bf16(kTile, kTile, false);
      int scores = 0, items = 0;  // Q K^T issued, items with chunks
      for (int k = 0; ok && next_work(k, w); ++k) {
        const Shape sh(w.it, p.tile_tokens);
        if (sh.most == 0) continue;
        wait(&bars.q_full, items);
        ++items;
        for (int j = sh.most - 1; j >= 0 && ok; --j, ++c) {
          const int slot = c % kSlots;
          wait(&bars.k_full[slot], c / kSlots);
#pragma unroll
          for (int s = 0; s < 2; ++s) {  // S = Q_s K_j^T, once the S before has been read
            if (j >= (s == 0 ? sh.n0 : sh.n1)) continue;
            if (scores > 0) wait(&bars.s_free, scores - 1);
            ++scores;
            if (!__all_sync(0xffffffffu, ok)) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              const uint64_t qd = ptx::sw128_desc(base + S::q + s * S::tile, 16, 1024);
              const uint64_t kd = ptx::sw128_desc(base + S::k + slot * S::tile, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32u;
                ptx::mma_ss(tmem, qd + (off >> 4), kd + (off >> 4), id_qk, kk > 0 ? 1u : 0u);
              }
              ptx::tc_commit(&bars.s_full[s]);
              if (s == 1 || sh.n1 == 0) {  // the chunk's last use
                ptx::tc_commit(&bars.k_empty[slot]);
                if (j == 0) ptx::tc_commit(&bars.q_empty);
              }
            }
            __syncwarp();
          }
          ok = __all_sync(0xffffffffu, ok);
        }
      }
    } else {
      constexpr uint32_t id_pv = ptx::idesc_bf16(kTile, D, true);
      int taken[2] = {0, 0};  // chunks of each tile so far
      for (int k = 0; ok && next_work(k, w); ++k) {
        const Shape sh(w.it, p.tile_tokens);
        for (int j = sh.most - 1; j >= 0 && ok; --j, ++c) {
          const int slot = c % kSlots;
          wait(&bars.v_ready[slot], c / kSlots);
#pragma unroll
          for (int s = 0; s < 2; ++s) {  // O_s += P_s V_j
            const int n = s == 0 ? sh.n0 : sh.n1;
            if (j >= n) continue;
            wait(&bars.p_full[s], taken[s]);
            ++taken[s];
            if (!__all_sync(0xffffffffu, ok)) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              const uint64_t vd = ptx::sw128_desc(base + S::v + slot * S::tile, kHalfBytes, 1024);
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                ptx::mma_ts(tmem + kTmO + s * D, tmem + kTmP + s * 64 + kk * 8,
                            vd + kk * (2048 >> 4), id_pv, (j < n - 1 || kk > 0) ? 1u : 0u);
              ptx::tc_commit(&bars.pv_done[s]);
              if (s == 1 || sh.n1 == 0) ptx::tc_commit(&bars.v_empty[slot]);
            }
            __syncwarp();
          }
          ok = __all_sync(0xffffffffu, ok);
        }
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
    // ------------------------------------------------------------ items, V guard
    set_regs_less();
    const uint32_t answer = ptx::smem_u32(&bars.answer);
    int c = 0, block = blockIdx.x;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Work w{};
      if (block >= 0) {
        w.it = p.a.tiles[block / p.a.kv_heads];
        w.hk = block % p.a.kv_heads;
        w.blocks = 1;
        if (!item_ok(p.a, w.it, 2 * p.tile_tokens)) {  // not the plan's: left out
          if (lane == 0) record_status(p.a.status, TLSP_ERR_DEVICE_ASSERT);
          w.it = PackedItem{0, 0, 0, 0, 0, 0, 0, -1};
        }
      }
      // the readers of item k - 2 are done with its place
      ok = k < 2 || ptx::mbar_wait(&bars.work_empty[k & 1], ((k >> 1) - 1) & 1, abort_flag, kWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) fail(bars, p.a.status);
        break;
      }
      if (lane == 0) {
        bars.work[k & 1] = w;
        ptx::mbar_arrive(&bars.work_full[k & 1]);
        if (w.blocks != 0) {  // ask for the next block meanwhile
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive_expect_tx(&bars.answer_full, 16);
          ptx::try_cancel(answer, &bars.answer_full);
        }
      }
      __syncwarp();
      if (w.blocks == 0) break;
      const Shape sh(w.it, p.tile_tokens);
      uint32_t* noted = bars.odd[k & 1];
      if (lane < 8) noted[lane] = 0;
      __syncwarp();
      for (int j = sh.most - 1; j >= 0; --j, ++c) {
        const int slot = c % kSlots;
        ok = ptx::mbar_wait(&bars.v_full[slot], (c / kSlots) & 1, abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) fail(bars, p.a.status);
          ok = false;
          break;
        }
        // chunk rows [0, every) are seen by all rows of the item, [every, some) by
        // part of them, the others by none
        int every, some;
        if (j < sh.pre) {
          every = some = min(kTile, w.it.pre_n - j * kTile);
        } else {
          const int at = (j - sh.pre) * kTile;
          some = min(kTile, sh.seen1 - at);
          every = min(some, max(0, w.it.diag + 1 - at));
        }
        if (every < kTile) {
          const uint32_t v = base + S::v + slot * S::tile;
          for (int h = 0; h < kHalves; ++h) {
            const uint32_t rows = v + h * kHalfBytes;  // 8 x 16 bytes a row
            const int end = some * 8;
            // eight pieces at a time; the usual answer is that all are finite
            for (int u = every * 8 + lane; u < end; u += 256) {
              uint4 x[8];
              uint32_t odd = 0;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[e] = u + 32 * e < end ? ptx::ld_shared_v4(rows + (u + 32 * e) * 16)
                                        : make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                odd |= exp_carry(x[e].x) | exp_carry(x[e].y) | exp_carry(x[e].z) | exp_carry(x[e].w);
              if (!(odd & 0x80008000u)) continue;
#pragma unroll 1
              for (int z = u; z < min(end, u + 256); z += 32) {
                const uint4 y = ptx::ld_shared_v4(rows + z * 16);
                const uint32_t m0 = odd_halves(y.x), m1 = odd_halves(y.y), m2 = odd_halves(y.z),
                               m3 = odd_halves(y.w);
                if (!(m0 | m1 | m2 | m3)) continue;
                ptx::st_shared_v4(rows + z * 16, y.x & ~m0, y.y & ~m1, y.z & ~m2, y.w & ~m3);
                const int bit = (j - sh.pre) * kTile + z / 8 - (w.it.diag + 1);
                atomicOr(&noted[bit >> 5], 1u << (bit & 31));
              }
            }
            for (int u = end + lane; u < kTile * 8; u += 32)
              ptx::st_shared_v4(rows + u * 16, 0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.v_ready[slot]);
      }
      // the answer lands before the shared memory goes away, even after an abort
      if (!ptx::mbar_wait(&bars.answer_full, k & 1, nullptr, kWaitNs)) {
        if (lane == 0) fail(bars, p.a.status);
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
      block = ptx::canceled_block(answer);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    set_regs_more();
    constexpr int kCols = D / 2;  // of O, for a thread
    // Where a thread stands. Built anew (from an opaque thread index) wherever the
    // chunk loop does not need it, so that it takes no registers there.
    struct Place {
      int s, half, r, i, gi;  // query tile, keys 64 half .. + 63 of a chunk, row, its token and head
      uint32_t tl;            // TMEM lanes
      __device__ __forceinline__ Place(const TileParams& p, uint32_t tmem) {
        int t;
        asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
        s = t >> 8;
        half = (t >> 7) & 1;
        r = t & 127;
        const int q = (int)(r * p.magic >> 16);
        i = q + s * p.tile_tokens;
        gi = r - q * p.a.group;
        tl = tmem + ((uint32_t)(r & ~31) << 16);
      }
      __device__ __forceinline__ uint32_t o_col() const { return tl + kTmO + s * D + half * kCols; }
      __device__ __forceinline__ bool real(const TileParams& p, const PackedItem& it) const {
        return r < p.tile_tokens * p.a.group && i < (s == 0 ? min(it.nt, p.tile_tokens) : it.nt);
      }
      // own keys that this row sees (spare rows: all)
      __device__ __forceinline__ int own_seen(const TileParams& p, const PackedItem& it) const {
        return real(p, it) ? max(0, min(it.kv_n, it.diag + i + 1)) : 0x7ffffe00;
      }
    };
    const int s = warp >> 3, half = (warp >> 2) & 1;
    const int pair = 1 + s * 4 + (warp & 3);  // barrier of the two warps of 32 rows
    const int all = 9 + s;                    // barrier of the tile's 256 threads
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = tl + 64 * half, p_col = tl + kTmP + s * 64 + 32 * half;
    int c = 0;  // chunks of this tile so far
    // After a failure a warp runs on (its partners wait for it at barriers; further
    // waits end soon), on whatever TMEM holds; nothing is written out then.
    auto wait = [&](uint64_t* bar, int parity) {
      if (!ptx::mbar_spin(bar, parity & 1, abort_flag, kWaitNs)) fail(bars, p.a.status);
      __syncwarp();
      ptx::tc_fence_after();
    };
    // The item stays in shared memory: what is needed of it now and then (masked
    // chunks, the epilogue) is read there, to keep registers for the scores.
    for (int k = 0;; ++k) {
      const Work& w = bars.work[k & 1];
      wait(&bars.work_full[k & 1], k >> 1);
      if (bar_or(all, 256, *abort_flag || w.blocks == 0)) break;
      const int c0 = c;
      int end, masked, ragged;  // up to end; before `masked`, and in `ragged`, some rows see part
      float m_run, l_run = 0.f;
      {
        const PackedItem it = w.it;
        const Shape sh(it, p.tile_tokens);
        const Place at(p, tmem);
        end = c0 + (s == 0 ? sh.n0 : sh.n1);
        const int whole = __reduce_min_sync(0xffffffffu, at.own_seen(p, it)) - 64 * half;
        masked = end - (sh.pre + max(0, whole + 64) / kTile);
        ragged = it.pre_n % kTile ? end - sh.pre : -1;
        m_run = at.real(p, it) ? -INFINITY : INFINITY;  // spare rows never raise it
      }
      for (; c < end; ++c) {
        wait(&bars.s_full[s], c);
        uint32_t x[2][32];  // the row's scores
        ptx::tmem_ld32(s_col, x[0]);
        ptx::tmem_ld32(s_col + 32, x[1]);
        ptx::tmem_ld_wait(x[0]);
        ptx::reg_barrier(x[1]);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.s_free);
        if (c < masked || c == ragged) {  // masked scores become -inf under either sign of the scale
          const PackedItem it = w.it;
          const int pre = (it.pre_n + kTile - 1) / kTile, j = end - 1 - c;
          const int seen = (j < pre ? it.pre_n - j * kTile
                                    : Place(p, tmem).own_seen(p, it) - (j - pre) * kTile) - 64 * half;
          const uint32_t off = p.scale_log2 < 0.f ? 0x7f800000u : 0xff800000u;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e >= seen) x[e / 32][e % 32] = off;
        }
        // their maximum (fmaxf drops a NaN; it comes back through ex2)
        float mx;
        if (p.scale_log2 >= 0.f) {
          float t[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            t[b] = __uint_as_float(x[b][0]);
#pragma unroll
            for (int e = 1; e + 1 < 32; e += 2)
              t[b] = ptx::max3(t[b], __uint_as_float(x[b][e]), __uint_as_float(x[b][e + 1]));
          }
          mx = fmaxf(ptx::max3(t[0], t[1], __uint_as_float(x[0][31])), __uint_as_float(x[1][31]));
        } else {
          mx = INFINITY;
#pragma unroll
          for (int e = 0; e < 64; ++e) mx = fminf(mx, __uint_as_float(x[e / 32][e % 32]));
        }
        mx *= p.scale_log2;
        // Raise the reference? The rows' two warps go together (TMEM accesses are
        // warp-collective); rows that need no raise move by less than 8.
        if (bar_or(pair, 64, mx > m_run + 8.f)) {
          // once P's columns are free the two threads of a row swap their maxima there
          if (c > c0) wait(&bars.pv_done[s], c - 1);
          ptx::tmem_st1(p_col, __float_as_uint(mx));
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          bar_sync(pair, 64);
          ptx::tc_fence_after();
          const float m_new =
              ptx::max3(m_run, mx, __uint_as_float(ptx::tmem_ld1(p_col + 32 - 64 * half)));
          if (c > c0) {  // O *= 2^(m_run - m_new)
            const float f = m_run == -INFINITY ? 0.f : ptx::ex2(m_run - m_new);
            const uint32_t o_col = Place(p, tmem).o_col();
#pragma unroll 1
            for (int q = 0; q < kCols / 8; ++q) {
              uint32_t o[8];
              ptx::tmem_ld8(o_col + q * 8, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              ptx::tmem_st8(o_col + q * 8, o);
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
        uint32_t pk[2][16];  // P, pairs of bf16
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const uint64_t y =
              ptx::f2_fma(ptx::f2_pack(__uint_as_float(x[e / 16][2 * (e % 16)]),
                                       __uint_as_float(x[e / 16][2 * (e % 16) + 1])),
                          sc2, nm2);
          float y0, y1;
          ptx::f2_unpack(y, y0, y1);
          const float p0 = ptx::ex2(y0), p1 = ptx::ex2(y1);
          sum2[e & 1] = ptx::f2_add(sum2[e & 1], ptx::f2_pack(p0, p1));
          pk[e / 16][e % 16] = pack_bf16(p0, p1);
        }
        if (c > c0) wait(&bars.pv_done[s], c - 1);  // the P before has been taken
        ptx::tmem_st16(p_col, pk[0]);
        ptx::tmem_st16(p_col + 16, pk[1]);
        float a0, a1, a2, a3;
        ptx::f2_unpack(sum2[0], a0, a1);
        ptx::f2_unpack(sum2[1], a2, a3);
        l_run += (a0 + a1) + (a2 + a3);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.p_full[s]);
      }
      const Place at(p, tmem);
      float* sums = reinterpret_cast<float*>(smem + S::sums) + at.s * 2 * kTile;
      const bool any = c > c0;
      if (any) {
        sums[at.half * kTile + at.r] = l_run;  // the halves of the row's sum
        wait(&bars.pv_done[s], c - 1);
      }
      if (bar_or(all, 256, *abort_flag != 0)) break;
      const PackedItem it = w.it;
      const bool real = at.real(p, it);
      const int half = at.half, i = at.i;
      const uint32_t o_col = at.o_col();
      const float l = any ? sums[at.r] + sums[kTile + at.r] : 0.f;
      const bool none = l == 0.f;  // no key seen
      const float inv = none ? 0.f : 1.f / l;
      const bool part = it.slot >= 0;
      const int head = w.hk * group + at.gi;
      if (real && half == 0) {
        const float lse = none ? -INFINITY : (m_run + log2f(l)) * kLn2;
        if (part)
          p.a.part_lse[(int64_t)(it.slot + i) * p.a.heads + head] = lse;
        else if (p.a.lse)
          p.a.lse[(int64_t)(it.q0 + i) * p.a.heads + head] = lse;
      }
      uint32_t any_odd = 0;
      if (any)
        for (int q = 0; q < 8; ++q) any_odd |= bars.odd[k & 1][q];
      // Each thread writes its half of the row from its registers, eight channels at a time:
      // wider steps, and rows staged in shared memory for stores of whole lines, cost
      // registers that the chunk loop then lacks (on a cool GPU, in turns: 24 ragged prompts
      // 201 us, 16384 tokens of 12 heads of 64 492 us; 16 channels: 201 and 536 us; staged:
      // 205 and 505 us. Back to back, at the power limit, the prompts take 237 us).
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.O.ptr) +
                           (int64_t)(it.q0 + i) * p.a.O.row_stride +
                           (int64_t)head * p.a.O.head_stride + half * kCols;
      float* part_out =
          p.a.part_o + ((int64_t)(it.slot + i) * p.a.heads + head) * D + half * kCols;
      __syncwarp();
#pragma unroll 1
      for (int q = 0; q < kCols; q += 8) {
        uint32_t o[8];
        if (any) ptx::tmem_ld8(o_col + q, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = none ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
        if (real && part) {
          uint4* to = reinterpret_cast<uint4*>(part_out + q);
          to[0] = make_uint4(o[0], o[1], o[2], o[3]);
          to[1] = make_uint4(o[4], o[5], o[6], o[7]);
        } else if (real) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = pack_bf16(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          *reinterpret_cast<uint4*>(out + q) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
      }
      if (any_odd) {
        // values that are not finite, of keys that only part of the rows see: added to
        // the rows that do, as written
#pragma unroll 1
        for (int q = 0; q < 256 && real; ++q) {
          if (!(bars.odd[k & 1][q >> 5] >> (q & 31) & 1) || q >= i) continue;  // key diag + 1 + q
          const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.a.V.ptr) +
                                   (int64_t)(it.kv0 + it.diag + 1 + q) * p.a.V.row_stride +
                                   w.hk * p.a.V.head_stride;
#pragma unroll 1
          for (int ch = 0; ch < kCols; ++ch) {
            const float z = __bfloat162float(v[half * kCols + ch]);
            if (fabsf(z) < INFINITY) continue;
            if (part)
              part_out[ch] += z;
            else
              out[ch] = __float2bfloat16_rn(__bfloat162float(out[ch]) + z);
          }
        }
      }
      ptx::tc_fence_before();  // O has been read before the next P is handed over
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.work_empty[k & 1]);
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
  p.magic = (65536u + a.group - 1) / a.group;
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
  return launch_dependent(kernel, dim3((unsigned)((int64_t)a.n_tiles * a.kv_heads)), kThreads,
                          (int)Smem<D>::bytes, 1, st, p);
}

}  // namespace

int packed_tile(const PackedArgs& a, cudaStream_t st) {
  return a.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace tlsp
