// Joins the partial results of rows whose keys were split over several items.
#include "packed.h"

namespace tlsp {
namespace {

// Partial results of a row over its key ranges: O = sum_p e^(lse_p - lse) O_p
// with lse = log sum_p e^(lse_p). One warp per row.
template <class T, int D>
__global__ void __launch_bounds__(256)
    packed_merge_kernel(const __grid_constant__ PackedArgs p) {
  const MergeItem it = p.merges[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + warp;
  if (row >= it.nt * p.heads) return;
  const int i = row / p.heads, h = row % p.heads;
  const int parts = it.a_parts + it.b_parts;
  const bool ok = it.q0 >= 0 && it.nt >= 1 && (int64_t)it.q0 + it.nt <= p.q_rows &&
                  it.a_parts >= 0 && it.b_parts >= 0 && it.a_slot >= 0 && it.b_slot >= 0 &&
                  it.a_stride >= 0 && it.b_stride >= 0 &&
                  (it.a_parts == 0 || it.a_slot + (int64_t)(it.a_parts - 1) * it.a_stride + it.nt <=
                                          p.part_rows) &&
                  (it.b_parts == 0 || it.b_slot + (int64_t)(it.b_parts - 1) * it.b_stride + it.nt <=
                                          p.part_rows);
  if (!ok) {
    if (lane == 0) record_status(p.status, TLSP_ERR_DEVICE_ASSERT);
    return;
  }
  auto part_row = [&](int q) {
    const int64_t slot = q < it.a_parts
                             ? it.a_slot + (int64_t)q * it.a_stride
                             : it.b_slot + (int64_t)(q - it.a_parts) * it.b_stride;
    return (slot + i) * p.heads + h;
  };
  float mx = -INFINITY;
  for (int q = lane; q < parts; q += 32) mx = fmaxf(mx, p.part_lse[part_row(q)]);
  mx = warp_max(mx);
  const float m_use = mx == -INFINITY ? 0.f : mx;
  constexpr int E = D / 32;
  float acc[E] = {};
  float sum = 0.f;
  for (int q0 = 0; q0 < parts; q0 += 32) {
    // a part that saw no key (lse -inf) has weight 0 and O = 0
    const float w_lane = q0 + lane < parts ? expf(p.part_lse[part_row(q0 + lane)] - m_use) : 0.f;
    const int n = min(32, parts - q0);
#pragma unroll 4
    for (int q = 0; q < n; ++q) {
      const float w = __shfl_sync(0xffffffffu, w_lane, q);
      const float* o = p.part_o + part_row(q0 + q) * D + lane * E;
      sum += w;
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4*>(o);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
        acc[2] = fmaf(w, v.z, acc[2]);
        acc[3] = fmaf(w, v.w, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(o);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
      }
    }
  }
  const bool none = sum == 0.f;
  const float inv = none ? 0.f : 1.f / sum;
  T* o = static_cast<T*>(p.O.ptr) + (it.q0 + i) * p.O.row_stride + h * p.O.head_stride + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = from_f32<T>(acc[e] * inv);
  if (p.lse && lane == 0)
    p.lse[(int64_t)(it.q0 + i) * p.heads + h] = none ? -INFINITY : m_use + logf(sum);
}

template <class T>
int merge(const PackedArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)a.n_merges, (unsigned)ceil_div((int64_t)kMergeTokens * a.heads, 8));
  if (grid.y > 65535) return TLSP_ERR_UNSUPPORTED;
  if (a.d == 128)
    packed_merge_kernel<T, 128><<<grid, 256, 0, st>>>(a);
  else
    packed_merge_kernel<T, 64><<<grid, 256, 0, st>>>(a);
  return check_launch();
}

}  // namespace

int packed_merge(const PackedArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? merge<__nv_bfloat16>(a, st) : merge<float>(a, st);
}

}  // namespace tlsp
