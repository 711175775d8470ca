// Rotary positions of queries and keys (forward and backward) in one launch.
//
// A pair (x1, x2) at position p becomes A (x1 cos a - x2 sin a, x2 cos a + x1
// sin a) with a = p w. The transposed map (the backward pass) turns by -a.
//
// Angles: the plan holds w / 2 pi modulo 1 as a 64-bit fraction F of a turn, so
// p F modulo 2^64 is the angle in turns, reduced exactly for every 64-bit
// position (the frequency's own rounding, 2^-65 of a turn, times p is the only
// error: 2^-34 of a turn at p = 2^31). Its top 32 bits as a signed number
// over 2^31 are the angle in half turns in [-1, 1), which sincospi takes.
//
// Bound: HBM; every element is read and written once. A thread owns the 16
// bytes (two pieces of 16 bytes with the half layout) of the same channels in
// several heads of one token, so sine and cosine are computed once for all of
// them; the heads are split over threads only as far as filling the GPU needs.
#include <cmath>

#include "kernels.h"

namespace tlsp {
namespace {

struct RotaryParams {
  tlsp_rotary_plan plan;
  const void* pos;
  int64_t pos_axis, pos_batch;
  int pos64;
  int batch, tokens;
  float sign;  // +1 forward, -1 backward
  tlsp_rotary_tensor t[2];
  int units;        // channel units of a head row (see rotary_kernel)
  int rot_units;    // of which the first rot_units are rotated
  int head_split;   // threads over which a token's heads are split
  int heads;        // t[0].heads + t[1].heads
};

// cos and sin (times the amplitude) of pair i at position index (b, n)
__device__ __forceinline__ void turn_of(const RotaryParams& p, int i, int b, int n, float& c,
                                        float& s) {
  const int64_t at = p.plan.axis[i] * p.pos_axis + b * p.pos_batch + n;
  const int64_t pos = p.pos64 ? reinterpret_cast<const int64_t*>(p.pos)[at]
                              : (int64_t) reinterpret_cast<const int32_t*>(p.pos)[at];
  const uint64_t turn = (uint64_t)pos * p.plan.turns[i];
  sincospif((float)(int32_t)(turn >> 32) * (1.f / 2147483648.f), &s, &c);
  c *= p.plan.amplitude;
  s *= p.plan.amplitude * p.sign;
}

template <class T>
struct Vec;  // 16 bytes of T
template <>
struct Vec<float> {
  static constexpr int n = 4;
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
};

// V consecutive elements to and from fp32: 16 bytes at a time where V says so
template <class T, int V>
__device__ __forceinline__ void load_n(const T* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = to_f32(p[0]);
  } else if constexpr (sizeof(T) == 4) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  } else {
    load8(p, x);
  }
}
template <class T, int V>
__device__ __forceinline__ void store_n(T* p, const float (&x)[V]) {
  if constexpr (V == 1) {
    p[0] = from_f32<T>(x[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = u;
  }
}

// One thread: unit u (channels) of token (b, n), heads h0, h0 + split, ...
// Units of V channels with the half layout: pieces [u V, u V + V) and
// [R/2 + u V, ...) for u < rot_units = R / 2 V; with the interleaved layout:
// 2 V' channels as one piece (V = Vec::n) or one pair (V = 1, two elements).
// Units behind rot_units copy one piece of V channels each.
template <class T, int V, bool kInter>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryParams p) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int u = (int)(id % p.units);
  const int64_t rest = id / p.units;
  const int part = (int)(rest % p.head_split);
  const int64_t row = rest / p.head_split;
  if (row >= (int64_t)p.batch * p.tokens) return;
  const int b = (int)(row / p.tokens), n = (int)(row % p.tokens);
  const int R = p.plan.rotary_dim, half = R / 2;
  constexpr int kPairs = kInter ? (V == 1 ? 1 : V / 2) : V;
  const bool turned = u < p.rot_units;

  float c[kPairs], s[kPairs];
  int at0, at1 = 0;  // channel offsets of the piece(s)
  if (turned) {
    const int i0 = u * kPairs;
#pragma unroll
    for (int e = 0; e < kPairs; ++e) turn_of(p, i0 + e, b, n, c[e], s[e]);
    at0 = kInter ? 2 * i0 : i0;
    at1 = half + i0;
  } else {
    at0 = R + (u - p.rot_units) * V;
  }
#pragma unroll 4
  for (int h = part; h < p.heads; h += p.head_split) {
    const bool second = h >= p.t[0].heads;
    const tlsp_rotary_tensor& t = p.t[second ? 1 : 0];
    const int hh = second ? h - p.t[0].heads : h;
    const T* in = static_cast<const T*>(t.in) + b * t.in_batch + n * t.in_token + hh * t.in_head;
    T* out = static_cast<T*>(t.out) + b * t.out_batch + n * t.out_token + hh * t.out_head;
    if (!turned) {
      float x[V];
      load_n<T, V>(in + at0, x);
      store_n<T, V>(out + at0, x);
    } else if constexpr (!kInter) {
      float x1[V], x2[V];
      load_n<T, V>(in + at0, x1);
      load_n<T, V>(in + at1, x2);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float y1 = fmaf(x1[e], c[e], -x2[e] * s[e]);
        x2[e] = fmaf(x2[e], c[e], x1[e] * s[e]);
        x1[e] = y1;
      }
      store_n<T, V>(out + at0, x1);
      store_n<T, V>(out + at1, x2);
    } else {
      constexpr int W = V == 1 ? 2 : V;
      float x[W];
      if constexpr (V == 1) {
        x[0] = to_f32(in[at0]);
        x[1] = to_f32(in[at0 + 1]);
      } else {
        load_n<T, V>(in + at0, x);
      }
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const float y1 = fmaf(x[2 * e], c[e], -x[2 * e + 1] * s[e]);
        x[2 * e + 1] = fmaf(x[2 * e + 1], c[e], x[2 * e] * s[e]);
        x[2 * e] = y1;
      }
      if constexpr (V == 1) {
        out[at0] = from_f32<T>(x[0]);
        out[at0 + 1] = from_f32<T>(x[1]);
      } else {
        store_n<T, V>(out + at0, x);
      }
    }
  }
}

bool wide_ok(const tlsp_rotary_tensor& t, int size, const tlsp_rotary_call& c) {
  const int64_t bytes[] = {t.in_token * size, t.in_head * size, t.out_token * size,
                           t.out_head * size, c.batch > 1 ? t.in_batch * size : 0,
                           c.batch > 1 ? t.out_batch * size : 0};
  for (int64_t b : bytes)
    if (b % 16 != 0) return false;
  return ((uintptr_t)t.in | (uintptr_t)t.out) % 16 == 0;
}

template <class T>
int launch(RotaryParams& p, const tlsp_rotary_call& call, bool two, cudaStream_t st) {
  constexpr int W = Vec<T>::n;
  const bool inter = p.plan.layout == TLSP_ROTARY_INTERLEAVED;
  const int R = p.plan.rotary_dim, d = p.plan.head_dim;
  bool wide = R % (inter ? W : 2 * W) == 0 && wide_ok(p.t[0], sizeof(T), call) &&
              (!two || wide_ok(p.t[1], sizeof(T), call));
  const int V = wide ? W : 1;
  p.rot_units = inter ? R / (wide ? W : 2) : R / 2 / V;
  // in place, the channels behind the rotated ones already hold their values
  const bool in_place = p.t[0].in == p.t[0].out && (!two || p.t[1].in == p.t[1].out);
  p.units = p.rot_units + (in_place ? 0 : (d - R) / V);
  const int64_t rows = (int64_t)p.batch * p.tokens;
  // Enough threads to fill the GPU (8 warps' worth per SM sub-partition), but no
  // more than that: each further split computes the angles once more.
  const int64_t want = (int64_t)device_sm_count() * 1024;
  int64_t split = std::min<int64_t>(p.heads, std::max<int64_t>(1, ceil_div(want, rows * p.units)));
  p.head_split = (int)split;
  const int64_t blocks = ceil_div(rows * p.units * split, 256);
  if (blocks > 0x7fffffffLL) return TLSP_ERR_UNSUPPORTED;
  auto go = [&](auto kernel) { kernel<<<(unsigned)blocks, 256, 0, st>>>(p); };
  if (wide)
    inter ? go(rotary_kernel<T, W, true>) : go(rotary_kernel<T, W, false>);
  else
    inter ? go(rotary_kernel<T, 1, true>) : go(rotary_kernel<T, 1, false>);
  return check_launch();
}

int validate_plan(const tlsp_rotary_plan* p) {
  if (!p) return TLSP_ERR_INVALID_ARG;
  if (p->head_dim < 8 || p->head_dim > 256 || p->head_dim % 8) return TLSP_ERR_INVALID_ARG;
  if (p->rotary_dim < 2 || p->rotary_dim > p->head_dim || p->rotary_dim % 2)
    return TLSP_ERR_INVALID_ARG;
  if (p->layout != TLSP_ROTARY_HALF && p->layout != TLSP_ROTARY_INTERLEAVED)
    return TLSP_ERR_INVALID_ARG;
  if (p->axes < 1 || p->axes > TLSP_ROTARY_MAX_AXES) return TLSP_ERR_INVALID_ARG;
  for (int i = 0; i < p->rotary_dim / 2; ++i)
    if (p->axis[i] >= p->axes) return TLSP_ERR_INVALID_ARG;
  return TLSP_OK;
}

int validate_tensor(const tlsp_rotary_tensor* t, int size) {
  if (!t->in || !t->out || t->heads < 1) return TLSP_ERR_INVALID_ARG;
  if ((uintptr_t)t->in % size || (uintptr_t)t->out % size) return TLSP_ERR_INVALID_ARG;
  if (t->in == t->out && (t->in_batch != t->out_batch || t->in_token != t->out_token ||
                          t->in_head != t->out_head))
    return TLSP_ERR_INVALID_ARG;
  return TLSP_OK;
}

}  // namespace
}  // namespace tlsp

using namespace tlsp;

extern "C" {

int tlsp_rotary_make_plan(const tlsp_rotary_desc* d, tlsp_rotary_plan* plan) {
  if (!d || !plan) return TLSP_ERR_INVALID_ARG;
  tlsp_rotary_plan p{};
  p.head_dim = d->head_dim;
  p.rotary_dim = d->rotary_dim;
  p.layout = d->layout;
  p.axes = d->axes;
  TLSP_TRY(validate_plan(&p));
  if (d->scaling < TLSP_ROTARY_NONE || d->scaling > TLSP_ROTARY_RAMP) return TLSP_ERR_INVALID_ARG;
  // written so that a NaN fails each check
  if (!(d->base > 0) || !std::isfinite(d->base)) return TLSP_ERR_INVALID_ARG;
  if (!(d->factor >= 1) || !std::isfinite(d->factor)) return TLSP_ERR_INVALID_ARG;
  if (!(d->amplitude >= 0) || !std::isfinite(d->amplitude)) return TLSP_ERR_INVALID_ARG;
  if (d->scaling == TLSP_ROTARY_RAMP &&
      (!(d->original_len > 0) || !std::isfinite(d->original_len) || !(d->slow >= 0) ||
       !(d->fast > d->slow) || !std::isfinite(d->fast)))
    return TLSP_ERR_INVALID_ARG;
  int64_t sum = 0;
  for (int a = 0; a < d->axes; ++a) {
    if (d->sections[a] < 0) return TLSP_ERR_INVALID_ARG;
    sum += d->sections[a];
  }
  if (sum != d->rotary_dim / 2) return TLSP_ERR_INVALID_ARG;
  p.amplitude = d->amplitude > 0 ? (float)d->amplitude
                : d->scaling == TLSP_ROTARY_RAMP ? (float)(1.0 + 0.1 * std::log(d->factor))
                                                 : 1.f;
  const double two_pi = 6.283185307179586476925286766559;
  int i = 0;
  for (int a = 0; a < d->axes; ++a) {
    const int s = d->sections[a];
    double base = d->base;
    if (d->scaling == TLSP_ROTARY_BASE && s > 1) base *= std::pow(d->factor, s / (s - 1.0));
    for (int e = 0; e < s; ++e, ++i) {
      double w = std::pow(base, -(double)e / s);
      if (d->scaling == TLSP_ROTARY_LINEAR) w /= d->factor;
      if (d->scaling == TLSP_ROTARY_RAMP) {
        const double r = (d->original_len * w / two_pi - d->slow) / (d->fast - d->slow);
        const double keep = std::fmin(1.0, std::fmax(0.0, r));
        w = keep * w + (1.0 - keep) * w / d->factor;
      }
      // whole turns do not matter at integer positions; long double keeps 64
      // bits of the fraction
      long double t = (long double)w / 6.283185307179586476925286766559005768L;
      t -= std::floor(t);
      long double f = std::nearbyint(t * 18446744073709551616.0L);
      p.turns[i] = f >= 18446744073709551616.0L ? 0 : (uint64_t)f;
      p.axis[i] = (uint8_t)a;
    }
  }
  *plan = p;
  return TLSP_OK;
}

int tlsp_rotary(const tlsp_rotary_plan* plan, const tlsp_rotary_call* call,
                const tlsp_rotary_tensor* Q, const tlsp_rotary_tensor* K, int32_t backward,
                void* stream) {
  TLSP_TRY(validate_plan(plan));
  if (!call || !Q || call->batch < 0 || call->tokens < 0 || (backward != 0 && backward != 1))
    return TLSP_ERR_INVALID_ARG;
  if (call->dtype != TLSP_F32 && call->dtype != TLSP_BF16) return TLSP_ERR_INVALID_ARG;
  if (call->batch == 0 || call->tokens == 0) return TLSP_OK;  // no rows: nothing to launch
  const int size = call->dtype == TLSP_BF16 ? 2 : 4;
  if (!call->positions || (uintptr_t)call->positions % (call->positions_64 ? 8 : 4))
    return TLSP_ERR_INVALID_ARG;
  TLSP_TRY(validate_tensor(Q, size));
  if (K) TLSP_TRY(validate_tensor(K, size));
  RotaryParams p{};
  p.plan = *plan;
  p.pos = call->positions;
  p.pos_axis = call->position_axis;
  p.pos_batch = call->position_batch;
  p.pos64 = call->positions_64 != 0;
  p.batch = call->batch;
  p.tokens = call->tokens;
  p.sign = backward ? -1.f : 1.f;
  p.t[0] = *Q;
  if (K) p.t[1] = *K;
  const int64_t heads = (int64_t)Q->heads + (K ? K->heads : 0);
  if (heads > 0x7fffffff) return TLSP_ERR_UNSUPPORTED;
  p.heads = (int)heads;
  cudaStream_t st = (cudaStream_t)stream;
  return call->dtype == TLSP_BF16 ? launch<__nv_bfloat16>(p, *call, K != nullptr, st)
                                  : launch<float>(p, *call, K != nullptr, st);
}

}  // extern "C"
