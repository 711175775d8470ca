// Joins the partial results of rows whose keys were split over several items:
//   O = sum_p e^(lse_p - lse) O_p with lse = log sum_p e^(lse_p).
//
// One warp per row, or, with many parts, a block (128 tokens of 2 heads behind a prefix in
// 118 parts, tile items and merge: 29 us with a warp, 24 with a block). Bound by latency
// (a few dependent reads of L2; 64 tokens x 40 heads of 128, 6 to 7 parts each: 6.8 us
// alone), so it starts while the kernel before is finishing, reads its item meanwhile (the
// other kernels of a call let the next one start only when what came before the call is
// done, so the table is there), and then has eight parts' rows in flight for a warp with
// their log partitions. fp32 throughout; parts are added in a fixed order, so results do
// not depend on which CTA was first.
#include "packed.h"

namespace tlsp {
namespace {

constexpr int kWarps = kMergeWarps, kAhead = kMergeAhead;

template <int D>
struct Row;  // a lane's channels of a row
template <>
struct Row<128> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void add(float w, float (&acc)[4]) const {
    acc[0] = fmaf(w, v.x, acc[0]);
    acc[1] = fmaf(w, v.y, acc[1]);
    acc[2] = fmaf(w, v.z, acc[2]);
    acc[3] = fmaf(w, v.w, acc[3]);
  }
};
template <>
struct Row<64> {
  float2 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ void add(float w, float (&acc)[2]) const {
    acc[0] = fmaf(w, v.x, acc[0]);
    acc[1] = fmaf(w, v.y, acc[1]);
  }
};

__device__ __forceinline__ void store(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store(float* p, const float (&x)[2]) {
  *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
}
template <int E>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(p + e) = __floats2bfloat162_rn(x[e], x[e + 1]);
}

// kJoint: the block's warps share a row's parts, else each takes a row.
template <class T, int D, bool kJoint>
__global__ void __launch_bounds__(32 * kWarps)
    packed_merge_kernel(const __grid_constant__ PackedArgs p) {
  const MergeItem it = p.merges[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = kJoint ? blockIdx.y : blockIdx.y * kWarps + warp;
  const int i = row / p.heads, h = row % p.heads;
  const int parts = it.a_parts + it.b_parts;
  const bool ok = it.q0 >= 0 && it.nt >= 1 && (int64_t)it.q0 + it.nt <= p.q_rows &&
                  it.a_parts >= 0 && it.b_parts >= 0 && it.a_slot >= 0 && it.b_slot >= 0 &&
                  it.a_stride >= 0 && it.b_stride >= 0 &&
                  (it.a_parts == 0 || it.a_slot + (int64_t)(it.a_parts - 1) * it.a_stride + it.nt <=
                                          p.part_rows) &&
                  (it.b_parts == 0 || it.b_slot + (int64_t)(it.b_parts - 1) * it.b_stride + it.nt <=
                                          p.part_rows);
  wait_for_previous();
  if (!ok) {
    if (threadIdx.x == 0) record_status(p.status, TLSP_ERR_DEVICE_ASSERT);
    return;
  }
  if (i >= it.nt) return;
  auto part_row = [&](int q) {
    const int64_t slot = q < it.a_parts
                             ? it.a_slot + (int64_t)q * it.a_stride
                             : it.b_slot + (int64_t)(q - it.a_parts) * it.b_stride;
    return (slot + i) * p.heads + h;
  };
  constexpr int E = D / 32;
  float acc[E] = {};
  float m = -INFINITY, sum = 0.f;  // running maximum of the log partitions
  const int first = kJoint ? (int)((int64_t)parts * warp / kWarps) : 0;
  const int last = kJoint ? (int)((int64_t)parts * (warp + 1) / kWarps) : parts;
  for (int q0 = first; q0 < last; q0 += 32) {  // 32 parts: a lane each for the weights
    const int n = min(32, last - q0);
    const float lse = lane < n ? p.part_lse[part_row(q0 + lane)] : -INFINITY;
    Row<D> rows[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (e < n) rows[e].load(p.part_o + part_row(q0 + e) * D + lane * E);
    const float to = fmaxf(m, warp_max(lse)), use = to == -INFINITY ? 0.f : to;
    const float f = m == -INFINITY ? 0.f : expf(m - use);
    m = to;
    sum *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
    // a part that saw no key (-inf) has weight 0, and O = 0
    const float w_lane = expf(lse - use);
    sum += warp_sum(w_lane);
    for (int b = 0; b < n; b += kAhead) {
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (b + e < n) {
          rows[e].add(__shfl_sync(0xffffffffu, w_lane, b + e), acc);
          if (b + e + kAhead < n) rows[e].load(p.part_o + part_row(q0 + b + e + kAhead) * D + lane * E);
        }
    }
  }
  if constexpr (kJoint) {
    __shared__ float s_acc[kWarps][D], s_m[kWarps], s_sum[kWarps];
#pragma unroll
    for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
    if (lane == 0) {
      s_m[warp] = m;
      s_sum[warp] = sum;
    }
    __syncthreads();
    if (warp != 0) return;
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w]);
    const float use = m == -INFINITY ? 0.f : m;
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = expf(s_m[w] - use);
      sum = fmaf(f, s_sum[w], sum);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(f, s_acc[w][lane * E + e], acc[e]);
    }
  }
  const bool none = sum == 0.f;
  const float inv = none ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] *= inv;
  store(static_cast<T*>(p.O.ptr) + (it.q0 + i) * p.O.row_stride + h * p.O.head_stride + lane * E, acc);
  if (p.lse && lane == 0)
    p.lse[(int64_t)(it.q0 + i) * p.heads + h] = none ? -INFINITY : m + logf(sum);
}

template <class T>
int merge(const PackedArgs& a, cudaStream_t st) {
  const bool joint = merge_joint(a.merge_parts);
  const int64_t blocks = merge_blocks(a.heads, a.merge_parts);
  if (blocks > kMaxGridY) return TLSP_ERR_UNSUPPORTED;  // (the planner refuses such plans)
  const dim3 grid((unsigned)a.n_merges, (unsigned)blocks);
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, 32 * kWarps, 0, 1, st, a); };
  if (joint) return a.d == 128 ? go(packed_merge_kernel<T, 128, true>) : go(packed_merge_kernel<T, 64, true>);
  return a.d == 128 ? go(packed_merge_kernel<T, 128, false>) : go(packed_merge_kernel<T, 64, false>);
}

}  // namespace

int packed_merge(const PackedArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? merge<__nv_bfloat16>(a, st) : merge<float>(a, st);
}

}  // namespace tlsp
