// gdn_rope kernel: rotary positions on the heads of q and k, forward and
// inverse (the gradient of a rotation is the rotation by the opposite angle).
//
//   angle_i = position * inv_freq[i],  i < rot / 2
//   (a, b) <- m (a cos - b sin, b cos + a sin)
// over the pairs (i, i + rot/2) of a head (half layout) or (2i, 2i + 1)
// (interleaved layout); elements from rot on pass through.
//
// Bound by the bytes of q and k, which neighbouring threads read and write in
// the order they lie in.  A thread has one piece of one head and forms its
// angles itself: no table of sines is read, and the arithmetic hides behind
// the bytes.  (Threads that take their piece of several heads share the
// angles among those but jump from head to head: 65536 tokens of 28 heads of
// 256 took 410 us with all heads a thread, 372 with four, 341 with one; fp32
// heads of 128 rotated whole 134, 119 and 117.)
// The angle is reduced in fp64 turns, position * inv_freq /
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

// This thread's token, head (the keys' behind the queries') and unit of the head.
struct Place {
  int64_t t;
  int unit;
  bool some;
  const void* src;
  void* dst;
};
template <typename T>
__device__ __forceinline__ Place place(const RopeParams& p) {
  Place w;
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x, row = id / (uint32_t)p.units, heads = (uint32_t)(p.h_q + p.h_k);
  const uint32_t t = row / heads, h = row - t * heads;
  w.unit = (int)(id - row * (uint32_t)p.units);
  w.t = t;
  w.some = t < p.tokens;
  const bool is_q = h < (uint32_t)p.h_q;
  const int64_t head = (int64_t)(is_q ? h : h - p.h_q) * p.d;
  w.src = reinterpret_cast<const T*>(is_q ? p.q : p.k) + w.t * (is_q ? p.q_stride : p.k_stride) + head;
  w.dst = reinterpret_cast<T*>(is_q ? p.q_out : p.k_out) + w.t * (is_q ? p.q_out_stride : p.k_out_stride) + head;
  return w;
}
__device__ __forceinline__ double position(const RopeParams& p, int64_t t) {
  return p.pos64 ? (double)reinterpret_cast<const int64_t*>(p.positions)[t] : (double)reinterpret_cast<const int32_t*>(p.positions)[t];
}
constexpr double kTurn = 0.15915494309189533577;  // 1 / 2 pi

// A unit is 2 N elements of a head: N of the first and N of the second half
// (half layout), 2 N neighbours (interleaved, and behind the rotated part).
template <typename T, int N, bool HALF>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p) {
  const Place w = place<T>(p);
  if (!w.some) return;
  const bool turned = w.unit < p.rot / (2 * N);
  // the unit's two spans
  const int a_at = turned && HALF ? w.unit * N : w.unit * 2 * N, b_at = turned && HALF ? p.rot / 2 + w.unit * N : a_at + N;
  const T* src = reinterpret_cast<const T*>(w.src);
  T* dst = reinterpret_cast<T*>(w.dst);
  float c[N], s[N];  // formed before the pieces are asked for: 342 us where asking first takes 350 (65536 tokens)
  if (turned) {
    const double pos = position(p, w.t);
    const float sign = p.inverse ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < N; ++i) turn<T>(pos * (p.inv_freq[w.unit * N + i] * kTurn), p.mscale, sign, c[i], s[i]);
  }
  Span<T, N> a = load_span<T, N>(src + a_at), b = load_span<T, N>(src + b_at);
  if (turned) {
    float x[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(a.v[i]), x[N + i] = to_f32(b.v[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int ia = HALF ? i : 2 * i, ib = HALF ? N + i : 2 * i + 1;
      const float u = x[ia], v = x[ib];
      x[ia] = u * c[i] - v * s[i];
      x[ib] = v * c[i] + u * s[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) a.v[i] = from_f32<T>(x[i]), b.v[i] = from_f32<T>(x[N + i]);
  }
  store_span<T, N>(dst + a_at, a);
  store_span<T, N>(dst + b_at, b);
}

// Any even rot and any d: one pair, or one element behind the rotated part, of kHeads heads, whose angle is the same
// (odd places leave nothing to load wide, and a thread of one head is bound by its angle and its place: 19016 tokens
// of 12 heads of 128, 66 of them rotated, 100 us, 41 with four).
constexpr int kHeads = 4;
template <typename T, bool HALF>
__global__ __launch_bounds__(kThreads) void rope_any_kernel(RopeParams p) {
  const int heads = p.h_q + p.h_k, parts = (heads + kHeads - 1) / kHeads;
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x, row = id / (uint32_t)p.units, t = row / (uint32_t)parts;
  const int unit = (int)(id - row * (uint32_t)p.units), first = (int)(row - t * (uint32_t)parts) * kHeads;
  if (t >= p.tokens) return;
  const bool turned = unit < p.rot / 2;
  const int a_at = !turned ? unit + p.rot / 2 : HALF ? unit : 2 * unit, b_at = !turned ? a_at : HALF ? unit + p.rot / 2 : a_at + 1;
  T u[kHeads], v[kHeads];
  T* dst[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = min(first + i, heads - 1);
    const bool is_q = h < p.h_q;
    const int64_t head = (int64_t)(is_q ? h : h - p.h_q) * p.d;
    const T* src = reinterpret_cast<const T*>(is_q ? p.q : p.k) + t * (is_q ? p.q_stride : p.k_stride) + head;
    dst[i] = reinterpret_cast<T*>(is_q ? p.q_out : p.k_out) + t * (is_q ? p.q_out_stride : p.k_out_stride) + head;
    u[i] = src[a_at], v[i] = src[b_at];
  }
  float c = 0.f, s = 0.f;
  if (turned) turn<T>(position(p, t) * (p.inv_freq[unit] * kTurn), p.mscale, p.inverse ? -1.f : 1.f, c, s);
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (first + i >= heads) break;
    if (turned) {
      const float x = to_f32(u[i]), y = to_f32(v[i]);
      dst[i][b_at] = from_f32<T>(y * c + x * s);
      u[i] = from_f32<T>(x * c - y * s);
    }
    dst[i][a_at] = u[i];
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
  const int64_t heads = p.h_q + p.h_k, per_token = (wide ? heads : (heads + kHeads - 1) / kHeads) * p.units;
  // thread numbers are 32-bit: a call of more runs its tokens in parts
  const int64_t most = ((int64_t)0xffffffff - kThreads) / per_token;
  if (p.tokens > most) {
    RopeParams a = p, b = p;
    a.tokens = most;
    b.tokens = p.tokens - most;
    b.positions = reinterpret_cast<const char*>(p.positions) + most * (p.pos64 ? 8 : 4);
    b.q = reinterpret_cast<const T*>(p.q) + most * p.q_stride;
    b.q_out = reinterpret_cast<T*>(p.q_out) + most * p.q_out_stride;
    if (p.h_k) b.k = reinterpret_cast<const T*>(p.k) + most * p.k_stride, b.k_out = reinterpret_cast<T*>(p.k_out) + most * p.k_out_stride;
    const hipError_t e = launch<T>(a, stream);
    return e != hipSuccess ? e : launch<T>(b, stream);
  }
  const dim3 grid((unsigned)((p.tokens * per_token + kThreads - 1) / kThreads));
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
