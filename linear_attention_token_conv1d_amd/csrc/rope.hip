// gdn_rope kernel: rotary positions on the heads of q and k, forward and
// inverse (the gradient of a rotation is the rotation by the opposite angle).
//
//   angle_i = position * inv_freq[i],  i < rot / 2
//   (a, b) <- m (a cos - b sin, b cos + a sin)
// over the pairs (i, i + rot/2) of a head (half layout) or (2i, 2i + 1)
// (interleaved layout); elements from rot on pass through.
//
// Bound by the bytes of q and k.  A thread owns the same elements of every
// head it visits: the angle is formed once for a token and pair and used for
// all of them, so the trigonometry costs next to nothing and no table of
// sines is read.  The angle is reduced in fp64 turns, position * inv_freq /
// 2 pi minus its nearest whole number, exact to 2^-53 of the unreduced angle
// (an fp32 product would be a tenth of a radian off at position 2^20).  Sine
// and cosine of the reduced turn are then fp32: the hardware's for bf16
// elements (error near 2^-20), sincospif for fp32 elements.
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void turn(double turns, float m, float sign, float& c, float& s);
template <>
__device__ __forceinline__ void turn<__bf16>(double turns, float m, float sign, float& c, float& s) {
  const float f = (float)(turns - rint(turns));
  c = m * __builtin_amdgcn_cosf(f);
  s = sign * m * __builtin_amdgcn_sinf(f);
}
template <>
__device__ __forceinline__ void turn<float>(double turns, float m, float sign, float& c, float& s) {
  const float f = (float)(turns - rint(turns));
  sincospif(2.f * f, &s, &c);
  c *= m;
  s *= sign * m;
}

template <typename T, int N>
struct alignas(sizeof(T) * N) Span {
  T v[N];
};
template <typename T, int N>
__device__ __forceinline__ Span<T, N> load_span(const T* p) {
  return *reinterpret_cast<const Span<T, N>*>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_span(T* p, const Span<T, N>& s) {
  *reinterpret_cast<Span<T, N>*>(p) = s;
}

// A unit is 2 N elements of a head: N of the first and N of the second half
// (half layout), 2 N neighbours (interleaved, and behind the rotated part).
// A thread takes one unit of one token in `per` heads of the nq + nk.
template <typename T, int N, bool HALF>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t job = id / p.units;  // token, then group of heads
  const int unit = (int)(id - job * p.units);
  const int64_t t = job / p.splits;
  if (t >= p.tokens) return;
  const int heads = p.h_q + p.h_k;
  int h = (int)(job - t * p.splits) * p.per;
  const int end = min(h + p.per, heads);
  const int rot_units = p.rot / (2 * N);
  const bool turned = unit < rot_units;
  // offsets of the unit's two spans inside a head
  const int a_at = turned ? (HALF ? unit * N : unit * 2 * N) : unit * 2 * N;
  const int b_at = turned && HALF ? p.rot / 2 + unit * N : a_at + N;
  float c[N], s[N];
  if (turned) {
    const double pos = p.pos64 ? (double)reinterpret_cast<const int64_t*>(p.positions)[t]
                               : (double)reinterpret_cast<const int32_t*>(p.positions)[t];
    const float sign = p.inverse ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      turn<T>(pos * (p.inv_freq[unit * N + i] * 0.15915494309189533577), p.mscale, sign, c[i], s[i]);
  }
#pragma unroll 4
  for (; h < end; ++h) {
    const bool is_q = h < p.h_q;
    const int64_t head = (int64_t)(is_q ? h : h - p.h_q) * p.d;
    const T* src = reinterpret_cast<const T*>(is_q ? p.q : p.k) + t * (is_q ? p.q_stride : p.k_stride) + head;
    T* dst = reinterpret_cast<T*>(is_q ? p.q_out : p.k_out) + t * (is_q ? p.q_out_stride : p.k_out_stride) + head;
    Span<T, N> a = load_span<T, N>(src + a_at), b = load_span<T, N>(src + b_at);
    if (turned) {
      float x[2 * N];
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = to_f32(a.v[i]), x[N + i] = to_f32(b.v[i]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int ia = HALF ? i : 2 * i, ib = HALF ? N + i : 2 * i + 1;
        const float u = x[ia], w = x[ib];
        x[ia] = u * c[i] - w * s[i];
        x[ib] = w * c[i] + u * s[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) a.v[i] = from_f32<T>(x[i]), b.v[i] = from_f32<T>(x[N + i]);
    }
    store_span<T, N>(dst + a_at, a);
    store_span<T, N>(dst + b_at, b);
  }
}

// Any even rot and any d: one pair, or one element behind the rotated part.
template <typename T, bool HALF>
__global__ __launch_bounds__(kThreads) void rope_any_kernel(RopeParams p) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t job = id / p.units;
  const int unit = (int)(id - job * p.units);
  const int64_t t = job / p.splits;
  if (t >= p.tokens) return;
  const int heads = p.h_q + p.h_k;
  int h = (int)(job - t * p.splits) * p.per;
  const int end = min(h + p.per, heads);
  const bool turned = unit < p.rot / 2;
  const int a_at = turned ? (HALF ? unit : 2 * unit) : unit + p.rot / 2;
  const int b_at = turned ? (HALF ? unit + p.rot / 2 : a_at + 1) : a_at;
  float c = 1.f, s = 0.f;
  if (turned) {
    const double pos = p.pos64 ? (double)reinterpret_cast<const int64_t*>(p.positions)[t]
                               : (double)reinterpret_cast<const int32_t*>(p.positions)[t];
    turn<T>(pos * (p.inv_freq[unit] * 0.15915494309189533577), p.mscale, p.inverse ? -1.f : 1.f, c, s);
  }
#pragma unroll 4
  for (; h < end; ++h) {
    const bool is_q = h < p.h_q;
    const int64_t head = (int64_t)(is_q ? h : h - p.h_q) * p.d;
    const T* src = reinterpret_cast<const T*>(is_q ? p.q : p.k) + t * (is_q ? p.q_stride : p.k_stride) + head;
    T* dst = reinterpret_cast<T*>(is_q ? p.q_out : p.k_out) + t * (is_q ? p.q_out_stride : p.k_out_stride) + head;
    const T a = src[a_at], b = src[b_at];
    if (turned) {
      const float u = to_f32(a), w = to_f32(b);
      dst[a_at] = from_f32<T>(u * c - w * s);
      dst[b_at] = from_f32<T>(w * c + u * s);
    } else {
      dst[a_at] = a;
    }
  }
}

bool spans_ok(const void* p, int64_t stride, int n, size_t es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (n * es) == 0 && stride % n == 0);
}

template <typename T>
hipError_t launch(RopeParams p, hipStream_t stream) {
  constexpr int N = 16 / (int)sizeof(T);
  const bool in_place = p.q == p.q_out && p.k == p.k_out;
  const bool wide = p.rot % (2 * N) == 0 && p.d % (2 * N) == 0 && spans_ok(p.q, p.q_stride, N, sizeof(T)) &&
                    spans_ok(p.k, p.k_stride, N, sizeof(T)) && spans_ok(p.q_out, p.q_out_stride, N, sizeof(T)) &&
                    spans_ok(p.k_out, p.k_out_stride, N, sizeof(T));
  // in place, what passes through stays where it is
  p.units = wide ? (in_place ? p.rot : p.d) / (2 * N) : (in_place ? p.rot / 2 : p.d - p.rot / 2);
  // heads to a thread: as many as leave the chip full (256 CUs of 2048 threads), to share the angles
  const int heads = p.h_q + p.h_k;
  int64_t splits = ((int64_t)256 * 2048 + p.tokens * p.units - 1) / (p.tokens * p.units);
  if (splits > heads) splits = heads;
  p.per = (int32_t)((heads + splits - 1) / splits);
  p.splits = (heads + p.per - 1) / p.per;
  const int64_t blocks = (p.tokens * p.splits * p.units + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  if (wide && p.half) hipLaunchKernelGGL((rope_kernel<T, N, true>), grid, dim3(kThreads), 0, stream, p);
  else if (wide) hipLaunchKernelGGL((rope_kernel<T, N, false>), grid, dim3(kThreads), 0, stream, p);
  else if (p.half) hipLaunchKernelGGL((rope_any_kernel<T, true>), grid, dim3(kThreads), 0, stream, p);
  else hipLaunchKernelGGL((rope_any_kernel<T, false>), grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeParams& p, int dtype, hipStream_t stream) {
  if (p.tokens == 0) return hipSuccess;
  return dtype == 1 ? launch<__bf16>(p, stream) : launch<float>(p, stream);
}

}  // namespace gdn
