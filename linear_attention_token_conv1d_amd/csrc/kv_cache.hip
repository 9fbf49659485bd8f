// gdn_cache_store kernel: new keys and values into the pages of an e4m3 cache
// with one scale for each (page, head).
//
//   scale = the least power of two with max |x| <= 448 scale over the page's
//           new tokens, and no less than the page's scale where it holds
//           tokens already;  code = e4m3(x / scale), to nearest even.
// With powers of two the division is exact, and where a page's scale grows
// its older codes are divided by the growth: exact again, but for values that
// fall among e4m3's subnormals.  (e4m3 keeps four bits at any size, so a scale
// between two powers of two would not make its values more exact.)
//
// One workgroup owns one (page, head) of the keys or the values, so the page's
// maximum, its scale and its older tokens need no atomics and no second
// launch.  Bound by bytes for long prompts (the values read, a code each
// written: 65536 tokens of 4 heads of 256 in 85 us, 4.8 TB/s, where a large copy
// reaches 5.1) and by latency for single tokens (6 us).  Keys lie [token][d] in a page,
// values [d][token]: attention then reads both with 16-byte loads in the order
// its matrix products take them.  Values are turned round through LDS.
#include "gdn_device.h"
#include "gdn_internal.h"
#include "sequences.h"

namespace gdn {
namespace {

constexpr float kMax = 448.f;  // largest e4m3 magnitude

// Four fp32 to four e4m3 codes: to nearest even, beyond the range to +-448, NaN to NaN.
__device__ __forceinline__ float clamp_code(float v) { return v != v ? v : fminf(fmaxf(v, -kMax), kMax); }
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_code(a), clamp_code(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_code(c), clamp_code(d), w, true);
}

// The least power of two s with v <= 448 s (448 = 1.75 * 2^8), at least 2^-126.
__device__ __forceinline__ float least_scale(float v) {
  const uint32_t u = __float_as_uint(v);
  int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

template <int THREADS>
__device__ __forceinline__ float block_max(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
  if constexpr (THREADS > 64) {
    __shared__ float s[THREADS / 64];
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int i = 1; i < THREADS / 64; ++i) v = fmaxf(v, s[i]);
  }
  return v;
}

// Which sequence a workgroup serves, and which of the pages that it writes to.
// Sequence n has the slots from cu[n] / page + 2 n on: at least as many as the
// pages that its tokens touch, wherever they begin.
__device__ __forceinline__ void find_slot(const CacheStoreParams& p, int slot, int& n, int& j) {
  if (!p.cu_seqlens) {
    n = slot / p.uniform_slots;
    j = slot - n * p.uniform_slots;
    return;
  }
  n = find_sequence(p.cu_seqlens, p.n_seqs, slot, [&](int64_t c, int i) { return c / p.page + 2 * (int64_t)i; });
  j = slot - (as_const(p.cu_seqlens)[n] / p.page + 2 * n);
}

// Four codes of a page whose scale grows, by the old scale over the new.
__device__ __forceinline__ uint32_t recode(uint32_t w, float ratio) {
  return encode4(__builtin_amdgcn_cvt_f32_fp8((int)w, 0) * ratio, __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * ratio,
                 __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * ratio, __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * ratio);
}
// The codes of a page's first `a` tokens, 16 at a time and four such pieces a thread on their way: in a decode step
// some page's scale grows nearly always, and the step waits for it (256 sequences, 4 heads of
// 256, whose pages all do: 31 us, 121 by single codes).  Slots
// from `a` on keep their bytes: no store covers them.
template <int THREADS>
__device__ __forceinline__ void recode_page(uint8_t* codes, int side, int a, int d, int page, float ratio, int tid) {
  const int pieces = side ? d * page / 16 : a * d / 16, row = page / 16 - 1;  // pieces of a row of values, less one
  for (int i0 = tid; i0 < pieces; i0 += THREADS * 4) {
    uint4 w[4];
    int n[4];  // of the piece's codes that belong to older tokens
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * THREADS;
      n[j] = i >= pieces ? 0 : side ? min(a - (i & row) * 16, 16) : 16;
      if (n[j] > 0) w[j] = *reinterpret_cast<const uint4*>(codes + i * 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n[j] <= 0) continue;
      uint8_t* at = codes + (i0 + j * THREADS) * 16;
      const uint32_t r[4] = {recode(w[j].x, ratio), recode(w[j].y, ratio), recode(w[j].z, ratio), recode(w[j].w, ratio)};
      if (n[j] == 16) {
        *reinterpret_cast<uint4*>(at) = make_uint4(r[0], r[1], r[2], r[3]);
      } else {
#pragma unroll
        for (int t = 0; t < 15; ++t)
          if (t < n[j]) at[t] = (uint8_t)(r[t >> 2] >> (8 * (t & 3)));
      }
    }
  }
}

// x / scale: by its reciprocal where that is exact, which it is for every scale but those that others have set.
struct Divide {
  float scale, inv;
  bool exact;
  __device__ __forceinline__ explicit Divide(float s) : scale(s), inv(1.f / s), exact((__float_as_uint(s) & 0x7fffffu) == 0) {}
  __device__ __forceinline__ float operator()(float x) const { return exact ? x * inv : x / scale; }
};

// The scale of a page whose new tokens reach `most` and whose older ones, if any, have the scale `was`.
__device__ __forceinline__ float page_scale(float most, float was) {
  const float least = least_scale(most);
  return was > least ? was : least;  // a scale that is not a number is replaced
}
__device__ __forceinline__ float magnitude(float x) {
  const float m = fabsf(x);
  return m < __builtin_inff() ? m : 0.f;  // NaN and infinities do not set the scale
}

// One new token a sequence: a wave for each (sequence, head, keys or values), E = D / 64 elements a lane, all in
// registers.  Bound by latency: the token is asked for before its page is known.
template <typename T, int D>
__global__ __launch_bounds__(256) void cache_store_one_kernel(CacheStoreParams p) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= (int64_t)p.n_seqs * p.h_kv * 2) return;
  const int side = (int)(unit & 1), n = (int)((unit >> 1) / p.h_kv), head = (int)((unit >> 1) - (int64_t)n * p.h_kv);
  const T* x = reinterpret_cast<const T*>(side ? p.v : p.k) + n * (side ? p.v_stride : p.k_stride) + head * D + lane * E;
  float f[E];
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = to_f32(x[e]);
  const int held = as_const(p.lens)[n];
  if (held < 0 || held / p.page >= p.max_pages) return;
  const int pid = as_const(p.page_table)[(int64_t)n * p.max_pages + held / p.page];
  if (pid < 0 || pid >= p.pages) return;
  const int a = held % p.page;
  float* scale_at = (side ? p.v_scale : p.k_scale) + (int64_t)pid * p.h_kv + head;
  const float was = a > 0 ? *scale_at : 0.f;
  float most = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) most = fmaxf(most, magnitude(f[e]));
  most = block_max<64>(most);
  const float scale = page_scale(most, was);
  const Divide by(scale);
  uint8_t* codes = (side ? p.v_cache : p.k_cache) + ((int64_t)pid * p.h_kv + head) * D * p.page;
  if (a > 0 && scale != was) recode_page<64>(codes, side, a, D, p.page, was / scale, lane);
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = by(f[e]);
  const uint32_t w = encode4(f[0], E > 1 ? f[E > 1 ? 1 : 0] : 0.f, E > 2 ? f[E > 2 ? 2 : 0] : 0.f, E > 3 ? f[E > 3 ? 3 : 0] : 0.f);
  uint8_t* at = codes + (side ? lane * E * p.page + a : a * D + lane * E);
  if (side) {
#pragma unroll
    for (int e = 0; e < E; ++e) at[e * p.page] = (uint8_t)(w >> (8 * e));
  } else if constexpr (E == 4) {
    *reinterpret_cast<uint32_t*>(at) = w;
  } else if constexpr (E == 2) {
    *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
  } else {
    *at = (uint8_t)w;
  }
  if (lane == 0) *scale_at = scale;
}

// Eight elements as they lie in memory, and the largest magnitude among them as an ordered whole number: two bf16 at a
// time, or fp32 bits.  Infinities and NaN are the largest of all, so a page without them shows that by its maximum.
template <typename T> struct Piece;
template <> struct alignas(16) Piece<__bf16> {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  static constexpr uint32_t kNotFinite = 0x7f800000u;
  uint32_t w[4];
  __device__ __forceinline__ float get(int e) const { return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]); }
  __device__ __forceinline__ void reach(uint32_t& most) const {
    u16x2 m = __builtin_bit_cast(u16x2, most);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    most = __builtin_bit_cast(uint32_t, m);
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t most) { return max(most << 16, most & 0xffff0000u); }  // as fp32
};
template <> struct alignas(16) Piece<float> {
  static constexpr uint32_t kNotFinite = 0x7f800000u;
  float v[8];
  __device__ __forceinline__ float get(int e) const { return v[e]; }
  __device__ __forceinline__ void reach(uint32_t& most) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t most) { return most; }
};

// Any number of new tokens: a workgroup for each (page, head, keys or values).  The values read for the maximum
// stay in registers up to kKeep pieces of 8 a thread (a page of 64 tokens of 256); what is beyond is read again.
constexpr int kKeep = 8;
template <typename T>
__global__ __launch_bounds__(256) void cache_store_kernel(CacheStoreParams p) {
  extern __shared__ uint8_t codes[];  // [tokens of the page][d + 4]: values only
  const int tid = threadIdx.x, head = blockIdx.y, side = blockIdx.z;
  int n, j;
  find_slot(p, blockIdx.x, n, j);
  const int64_t begin = p.cu_seqlens ? max(as_const(p.cu_seqlens)[n], 0) : (int64_t)n * p.uniform;
  const int64_t end = p.cu_seqlens ? min((int64_t)as_const(p.cu_seqlens)[n + 1], p.tokens) : begin + p.uniform;
  const int64_t held = as_const(p.lens)[n];  // tokens of the sequence in the cache
  if (held < 0 || end <= begin || j < 0) return;  // (slots ahead of a pack that does not begin at token 0)
  const int64_t first = (held / p.page + j) * p.page;  // the page's first position
  if (first >= held + (end - begin) || first / p.page >= p.max_pages) return;
  // slots [a, b) of the page get the tokens from row on
  const int a = (int)max(held - first, (int64_t)0);
  const int b = (int)min(held + (end - begin) - first, (int64_t)p.page);
  const int64_t row = begin + first + a - held;
  const int d = p.d, shift = d == 256 ? 5 : d == 128 ? 4 : 3, per = d / 8;  // pieces of 8 elements, 2^shift a token
  const int count = (b - a) * per;
  const T* x = reinterpret_cast<const T*>(side ? p.v : p.k) + row * (side ? p.v_stride : p.k_stride) + head * d;
  const int64_t stride = side ? p.v_stride : p.k_stride;
  auto load = [&](int i) { return *reinterpret_cast<const Piece<T>*>(x + (i >> shift) * stride + (i & (per - 1)) * 8); };
  Piece<T> kept[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (tid + 256 * k < count) kept[k] = load(tid + 256 * k);
  const int pid = as_const(p.page_table)[(int64_t)n * p.max_pages + first / p.page];
  if (pid < 0 || pid >= p.pages) return;
  float* scale_at = (side ? p.v_scale : p.k_scale) + (int64_t)pid * p.h_kv + head;
  const float was = a > 0 ? *scale_at : 0.f;

  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (tid + 256 * k < count) kept[k].reach(bits);
  for (int i = tid + 256 * kKeep; i < count; i += 256) load(i).reach(bits);
  // (whole numbers below 2^31 keep their order as fp32 bits, but NaN's would not: they go by their own flag)
  bits = Piece<T>::bits(bits);
  const bool wild = __syncthreads_or(bits >= Piece<T>::kNotFinite);
  if (wild) {  // infinities and NaN do not set the scale
    float most = 0.f;
    for (int i = tid; i < count; i += 256) {
      const Piece<T> f = load(i);
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, magnitude(f.get(e)));
    }
    bits = __float_as_uint(most);
  }
  const float scale = page_scale(block_max<256>(__uint_as_float(bits)), was);
  const Divide by(scale);
  uint8_t* out = (side ? p.v_cache : p.k_cache) + ((int64_t)pid * p.h_kv + head) * d * p.page;

  if (a > 0 && scale != was) recode_page<256>(out, side, a, d, p.page, was / scale, tid);
  auto put = [&](int i, const Piece<T>& piece) {
    float f[8];
    uint32_t lo, hi;
    if (!wild && by.exact) {  // all within the range
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = piece.get(e) * by.inv;
      lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false), true);
      hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false), true);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = by(piece.get(e));
      lo = encode4(f[0], f[1], f[2], f[3]), hi = encode4(f[4], f[5], f[6], f[7]);
    }
    const int t = i >> shift, c = (i & (per - 1)) * 8;
    if (side) {
      uint32_t* at = reinterpret_cast<uint32_t*>(codes + t * (d + 4) + c);
      at[0] = lo;
      at[1] = hi;
    } else {
      *reinterpret_cast<uint2*>(out + (a + t) * d + c) = make_uint2(lo, hi);
    }
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (tid + 256 * k < count) put(tid + 256 * k, kept[k]);
  for (int i = tid + 256 * kKeep; i < count; i += 256) put(i, load(i));
  __syncthreads();  // every thread has read the page's scale; the values' codes are in LDS
  if (tid == 0) *scale_at = scale;
  if (!side) return;
  // Values turned round: a thread takes 4 elements of 16 neighbouring slots, 16 words from LDS, and turns them 4 by
  // 4 bytes; neighbouring threads have an element's next slots, so that they write whole rows of a page together.
  // Rows of d + 4 bytes keep their reads in different banks.
  const int g0 = a / 16, groups = (b + 15) / 16 - g0;
  for (int i = tid; i < groups * (d / 4); i += 256) {
    const int c = i / groups * 4, s0 = (g0 + i % groups) * 16;
    uint8_t* at = out + c * p.page + s0;
    if (s0 >= a && s0 + 16 <= b) {
      uint32_t r[4][4];  // [element][slots / 4]
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t*>(codes + (s0 - a + 4 * q + e) * (d + 4) + c);
        // 4 x 4 bytes: first and second halves of the words' pairs, then their bytes
        const uint32_t p0 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400), p1 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400);
        const uint32_t p2 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602), p3 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
        r[0][q] = __builtin_amdgcn_perm(p1, p0, 0x05040100);
        r[1][q] = __builtin_amdgcn_perm(p1, p0, 0x07060302);
        r[2][q] = __builtin_amdgcn_perm(p3, p2, 0x05040100);
        r[3][q] = __builtin_amdgcn_perm(p3, p2, 0x07060302);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4*>(at + e * p.page) = make_uint4(r[e][0], r[e][1], r[e][2], r[e][3]);
    } else {
      for (int t = max(0, a - s0); t < min(16, b - s0); ++t) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + (s0 - a + t) * (d + 4) + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) at[e * p.page + t] = (uint8_t)(w >> (8 * e));
      }
    }
  }
}

template <typename T>
hipError_t launch(CacheStoreParams p, hipStream_t stream) {
  int64_t slots;
  if (p.cu_seqlens) {
    slots = p.tokens / p.page + 2 * (int64_t)p.n_seqs;
  } else {
    p.uniform = p.tokens / p.n_seqs;
    p.uniform_slots = (int32_t)((p.uniform + p.page - 2) / p.page + 1);
    slots = (int64_t)p.uniform_slots * p.n_seqs;
    if (p.uniform == 1) {
      const dim3 grid((unsigned)(((int64_t)p.n_seqs * p.h_kv * 2 + 3) / 4));
      if (p.d == 64) hipLaunchKernelGGL((cache_store_one_kernel<T, 64>), grid, dim3(256), 0, stream, p);
      else if (p.d == 128) hipLaunchKernelGGL((cache_store_one_kernel<T, 128>), grid, dim3(256), 0, stream, p);
      else hipLaunchKernelGGL((cache_store_one_kernel<T, 256>), grid, dim3(256), 0, stream, p);
      return hipGetLastError();
    }
  }
  const size_t lds = (size_t)p.page * (p.d + 4);
  hipLaunchKernelGGL((cache_store_kernel<T>), dim3((unsigned)slots, (unsigned)p.h_kv, 2), dim3(256), lds, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_store(const CacheStoreParams& p, int dtype, hipStream_t stream) {
  if (p.tokens == 0) return hipSuccess;
  return dtype == 1 ? launch<__bf16>(p, stream) : launch<float>(p, stream);
}

}  // namespace gdn
