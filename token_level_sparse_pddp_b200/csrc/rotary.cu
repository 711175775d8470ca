// Rotary positions of queries and keys (forward and backward) in one launch.
//
// A pair (x1, x2) at position p becomes A (x1 cos a - x2 sin a, x2 cos a + x1
// sin a) with a = p w. The transposed map (the backward pass) turns by -a.
//
// Angles: the plan holds w / 2 pi modulo 1 as a 64-bit fraction F of a turn, so
// p F modulo 2^64 is the angle in turns, reduced without an error of its own for every
// 64-bit position. Its top 32 bits as a signed number over 2^31 are the angle in half
// turns in [-1, 1), which sincospi takes. What is off: F by up to 2^-56 of a turn (w is a
// 64-bit floating-point number), which counts p times: 2^-25 of a turn at p = 2^31; and,
// at every position, the rounding of those 32 bits to fp32's 24: up to 2^-26 of a turn.
//
// Bound: HBM; every element is read and written once. A thread owns two 16-byte
// pieces of a head row (with the half layout the two halves of its pairs) and goes
// through the heads of one token with them, so sine and cosine are computed once for
// all of them. It loads the pieces of a batch of heads before it writes the first: in
// and out may be the same memory, so the compiler cannot do that by itself. The heads
// are split over threads only as far as filling the GPU needs.
// Measured on replay (12 + 12 heads x 32760 tokens x 128, bf16, 403 MB): 65.8 us = 6.1
// TB/s with batches of two heads, 71 with four (fewer threads fit), 73 without batches.
// fp32 (2 x 24 heads x 4680 x 64, 115 MB): 18.2 us = 6.3 TB/s with four, 19.6 with two,
// 23.8 without: 16 bytes hold half as many pairs, so angles and registers weigh half as
// much.
#include <cmath>

#include "kernels.h"
#include "overlap.h"

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
  int units;       // threads of a head row, of which the first rot_units turn
  int rot_units;
  int pieces;      // pieces of the rotated channels (interleaved layout), of the others
  int rest;
  int head_split;  // threads over which a token's batches of heads are split
  int batches[2];  // of heads, of the two tensors
};

template <class T>
constexpr int kBatch = sizeof(T) == 2 ? 2 : 4;  // heads loaded at once
constexpr int kThreads = 128;

// The plan lies among the kernel's parameters, from where lanes that read different
// entries get them one after the other. Through an address whose origin the compiler does
// not see they come like global memory (37762 tokens of 3 + 1 heads of 128: 14.1 us, 15.1
// the other way; the case above 65.8 and 67.0).
template <class E>
__device__ __forceinline__ const E* as_memory(const E* p) {
  asm volatile("" : "+l"(p));
  return p;
}

// cos and sin (times the amplitude) of pairs i .. i + V - 1 (the first `count` are used) at
// position index (b, n)
template <int V>
__device__ __forceinline__ void turns_of(const RotaryParams& p, int i, int count, int b, int n,
                                         float (&c)[V], float (&s)[V]) {
  const uint64_t* turns = as_memory(p.plan.turns) + i;
  const uint8_t* axis = as_memory(p.plan.axis) + i;
  const int64_t at = b * p.pos_batch + n;
  auto position = [&](int64_t x) {
    return p.pos64 ? reinterpret_cast<const int64_t*>(p.pos)[x]
                   : (int64_t) reinterpret_cast<const int32_t*>(p.pos)[x];
  };
  const bool one = p.plan.axes == 1;
  const int64_t first = one ? position(at) : 0;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (e >= count) break;
    const int64_t pos = one ? first : position(axis[e] * p.pos_axis + at);
    const uint64_t turn = (uint64_t)pos * turns[e];
    sincospif((float)(int32_t)(turn >> 32) * (1.f / 2147483648.f), &s[e], &c[e]);
    c[e] *= p.plan.amplitude;
    s[e] *= p.plan.amplitude * p.sign;
  }
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

// V consecutive elements as they lie in memory: one element, or 16 bytes.
template <class T, int V>
struct Piece {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = to_f32(v); }
  __device__ __forceinline__ void set(const float (&x)[1]) { v = from_f32<T>(x[0]); }
};
template <>
struct Piece<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  __device__ __forceinline__ void set(const float (&x)[4]) { v = make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Piece<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  }
};

// (x1, x2) turned: fp32, one rounding per product-sum
__device__ __forceinline__ void turn(float& x1, float& x2, float c, float s) {
  const float y1 = fmaf(x1, c, -x2 * s);
  x2 = fmaf(x2, c, x1 * s);
  x1 = y1;
}

// One thread: unit u of token (b, n), batches of heads part, part + split, ... A unit is
// two pieces of V channels at c0 and c1 (the second may be missing): with the half
// layout channel c0 + e pairs with c1 + e, with the interleaved one neighbours within
// a piece do (V = 1: c0 with c1 in both). Units behind rot_units copy.
// (bf16: 64 registers, for the threads that hide the reads; fp32 is slower with that: 19.5
// us instead of 18.2.)
template <class T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 1) rotary_kernel(const __grid_constant__ RotaryParams p) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int u = (int)(id % p.units);
  const int64_t rest = id / p.units;
  const int part = (int)(rest % p.head_split);
  const int64_t row = rest / p.head_split;
  if (row >= (int64_t)p.batch * p.tokens) {
    wait_for_previous();
    return;
  }
  const int b = (int)(row / p.tokens), n = (int)(row % p.tokens);
  const int R = p.plan.rotary_dim;
  const bool turned = u < p.rot_units;
  wait_for_previous();

  float c[V], s[V];
  int c0, c1;
  bool two = true;
  if (turned) {
    if (kInter && V > 1) {
      c0 = 2 * u * V;
      c1 = c0 + V;
      two = 2 * u + 1 < p.pieces;
    } else {
      c0 = kInter ? 2 * u : u * V;
      c1 = kInter ? c0 + 1 : R / 2 + c0;
    }
    turns_of<V>(p, u * V, two ? V : V / 2, b, n, c, s);
  } else {
    c0 = R + 2 * (u - p.rot_units) * V;
    c1 = c0 + V;
    two = 2 * (u - p.rot_units) + 1 < p.rest;
  }
  for (int q = part; q < p.batches[0] + p.batches[1]; q += p.head_split) {
    const bool second = q >= p.batches[0];
    const tlsp_rotary_tensor& t = p.t[second ? 1 : 0];
    constexpr int B = kBatch<T>;
    const int h0 = (second ? q - p.batches[0] : q) * B, count = min(B, t.heads - h0);
    const T* in = static_cast<const T*>(t.in) + b * t.in_batch + n * t.in_token + h0 * t.in_head;
    T* out = static_cast<T*>(t.out) + b * t.out_batch + n * t.out_token + h0 * t.out_head;
    Piece<T, V> x[B][2];
#pragma unroll
    for (int h = 0; h < B; ++h) {
      if (h >= count) break;
      x[h][0].load(in + h * t.in_head + c0);
      if (two) x[h][1].load(in + h * t.in_head + c1);
    }
#pragma unroll
    for (int h = 0; h < B; ++h) {
      if (h >= count) break;
      if (turned) {
        float a[V], d[V];
        x[h][0].get(a);
        x[h][1].get(d);
        if constexpr (kInter && V > 1) {
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            turn(a[2 * e], a[2 * e + 1], c[e], s[e]);
            turn(d[2 * e], d[2 * e + 1], c[V / 2 + e], s[V / 2 + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) turn(a[e], d[e], c[e], s[e]);
        }
        x[h][0].set(a);
        x[h][1].set(d);
      }
      x[h][0].store(out + h * t.out_head + c0);
      if (two) x[h][1].store(out + h * t.out_head + c1);
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
  p.pieces = R / V;
  p.rot_units = (int)ceil_div(p.pieces, 2);
  // in place, the channels behind the rotated ones already hold their values
  const bool in_place = p.t[0].in == p.t[0].out && (!two || p.t[1].in == p.t[1].out);
  p.rest = in_place ? 0 : (d - R) / V;
  p.units = p.rot_units + (int)ceil_div(p.rest, 2);
  p.batches[0] = (int)ceil_div(p.t[0].heads, kBatch<T>);
  p.batches[1] = two ? (int)ceil_div(p.t[1].heads, kBatch<T>) : 0;
  const int64_t rows = (int64_t)p.batch * p.tokens;
  // Enough threads to fill the GPU, but no more than that: each further split computes the
  // angles once more (bf16, 37762 tokens of 3 + 1 heads: 14.1 us, 24.7 with 4096 threads an
  // SM; the case above 65.8 us with 1536, 74.8 with 8192; 16381 tokens of 40 + 8 heads 66.3
  // us, 78 with 768. fp32, the case above: 18.2 us with 1024, 19.2 with 768, 22.7 with 2048).
  const int64_t want = (int64_t)device_sm_count() * (sizeof(T) == 2 ? 1536 : 1024);
  const int64_t split = std::min<int64_t>(p.batches[0] + p.batches[1],
                                          std::max<int64_t>(1, ceil_div(want, rows * p.units)));
  p.head_split = (int)split;
  const int64_t blocks = ceil_div(rows * p.units * split, kThreads);
  if (blocks > 0x7fffffffLL) return TLSP_ERR_UNSUPPORTED;
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, dim3((unsigned)blocks), kThreads, 0, 1, st, p);
  };
  if (wide) return inter ? go(rotary_kernel<T, W, true>) : go(rotary_kernel<T, W, false>);
  return inter ? go(rotary_kernel<T, 1, true>) : go(rotary_kernel<T, 1, false>);
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
  return TLSP_OK;
}

// A thread writes its heads of a token while others still read theirs: an output shares
// memory with its own input only if it is that input, else with no input and no output, and
// its own elements lie apart.
int validate_overlap(const RotaryParams& p, int count, int size) {
  auto span = [&](const void* at, int64_t batch, int64_t token, int64_t head, int heads) {
    return Span(at, (int64_t)p.plan.head_dim * size)
        .with(p.batch, (__int128)batch * size)
        .with(p.tokens, (__int128)token * size)
        .with(heads, (__int128)head * size);
  };
  auto in = [&](const tlsp_rotary_tensor& t) {
    return span(t.in, t.in_batch, t.in_token, t.in_head, t.heads);
  };
  auto out = [&](const tlsp_rotary_tensor& t) {
    return span(t.out, t.out_batch, t.out_token, t.out_head, t.heads);
  };
  for (int x = 0; x < count; ++x) {
    const tlsp_rotary_tensor& t = p.t[x];
    const Span o = out(t);
    if (!o.distinct()) return TLSP_ERR_INVALID_ARG;
    const bool in_place = t.in == t.out && (p.batch == 1 || t.in_batch == t.out_batch) &&
                          (p.tokens == 1 || t.in_token == t.out_token) &&
                          (t.heads == 1 || t.in_head == t.out_head);
    if (!in_place && !apart(o, in(t))) return TLSP_ERR_INVALID_ARG;
    if (count == 2 && (!apart(o, in(p.t[1 - x])) || !apart(o, out(p.t[1 - x]))))
      return TLSP_ERR_INVALID_ARG;
  }
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
  TLSP_TRY(validate_overlap(p, K ? 2 : 1, size));
  cudaStream_t st = (cudaStream_t)stream;
  return call->dtype == TLSP_BF16 ? launch<__nv_bfloat16>(p, *call, K != nullptr, st)
                                  : launch<float>(p, *call, K != nullptr, st);
}

}  // extern "C"
