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
// One workgroup owns one (page, head) of the keys or the values, so the
// page's maximum, its scale and its older tokens need no atomics and no second
// launch.  Bound by bytes for long prompts (the values read, a code each
// written) and by latency for single tokens.  Keys lie [token][d] in a page,
// values [d][token]: attention then reads both with 16-byte loads in the order
// its matrix products take them.  Values are turned round through LDS.
#include "gdn_device.h"
#include "gdn_internal.h"

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
  cint32* cu = as_const(p.cu_seqlens);
  int lo = 0, hi = p.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] / p.page + 2 * mid <= slot) lo = mid; else hi = mid - 1;
  }
  n = lo;
  j = slot - (cu[lo] / p.page + 2 * lo);
}

template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void cache_store_kernel(CacheStoreParams p) {
  extern __shared__ uint8_t codes[];  // [tokens of the page][d]: values only
  const int tid = threadIdx.x, head = blockIdx.y, side = blockIdx.z;
  int n, j;
  find_slot(p, blockIdx.x, n, j);
  const int64_t begin = p.cu_seqlens ? max(as_const(p.cu_seqlens)[n], 0) : (int64_t)n * p.uniform;
  const int64_t end = p.cu_seqlens ? min((int64_t)as_const(p.cu_seqlens)[n + 1], p.tokens) : begin + p.uniform;
  const int64_t held = as_const(p.lens)[n];  // tokens of the sequence in the cache
  if (held < 0 || end <= begin) return;
  const int64_t first = (held / p.page + j) * p.page;  // the page's first position
  if (first >= held + (end - begin) || first / p.page >= p.max_pages) return;
  const int pid = as_const(p.page_table)[(int64_t)n * p.max_pages + first / p.page];
  if (pid < 0 || pid >= p.pages) return;
  // slots [a, b) of the page get the tokens from row on
  const int a = (int)max(held - first, (int64_t)0);
  const int b = (int)min(held + (end - begin) - first, (int64_t)p.page);
  const int64_t row = begin + first + a - held;
  const int d = p.d, per = d / 8;  // 8 elements a thread
  const T* x = reinterpret_cast<const T*>(side ? p.v : p.k) + row * (side ? p.v_stride : p.k_stride) + head * d;
  const int64_t stride = side ? p.v_stride : p.k_stride;

  float most = 0.f;
  for (int i = tid; i < (b - a) * per; i += THREADS) {
    const int t = i / per, c = (i - t * per) * 8;
    float f[8];
    load8(x + t * stride + c, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = fabsf(f[e]);
      most = fmaxf(most, m < __builtin_inff() ? m : 0.f);  // NaN and infinities do not set the scale
    }
  }
  float* scale_at = (side ? p.v_scale : p.k_scale) + (int64_t)pid * p.h_kv + head;
  const float was = a > 0 ? *scale_at : 0.f;
  most = block_max<THREADS>(most);
  const float least = least_scale(most);
  const float scale = was > least ? was : least;  // a scale that is not a number is replaced
  const float inv = 1.f / scale;  // exact, unless the page's scale was set by others
  uint8_t* out = (side ? p.v_cache : p.k_cache) + ((int64_t)pid * p.h_kv + head) * d * p.page;

  if (a > 0 && scale != was) {  // the page's older tokens, by the new scale
    const float ratio = was * inv;
    for (int i = tid; i < a * d; i += THREADS) {
      const int t = i / d, c = i - t * d;
      uint8_t* at = out + (side ? c * p.page + t : i);
      const float old = __builtin_amdgcn_cvt_f32_fp8((int)*at, 0);
      *at = (uint8_t)encode4(old * ratio, 0.f, 0.f, 0.f);
    }
  }
  for (int i = tid; i < (b - a) * per; i += THREADS) {
    const int t = i / per, c = (i - t * per) * 8;
    float f[8];
    load8(x + t * stride + c, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    uint2 w;
    w.x = encode4(f[0], f[1], f[2], f[3]);
    w.y = encode4(f[4], f[5], f[6], f[7]);
    *reinterpret_cast<uint2*>(side ? codes + t * d + c : out + (int64_t)(a + t) * d + c) = w;
  }
  __syncthreads();
  if (tid == 0) *scale_at = scale;
  if (!side) return;
  // values: 16 neighbouring slots of one element a turn, bytes where the new tokens end inside them
  const int g0 = a / 16, groups = (b + 15) / 16 - g0;
  for (int i = tid; i < groups * d; i += THREADS) {
    const int c = i % d, s0 = (g0 + i / d) * 16;
    uint8_t* at = out + (int64_t)c * p.page + s0;
    if (s0 >= a && s0 + 16 <= b) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        w[q] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[q] |= (uint32_t)codes[(s0 - a + 4 * q + e) * d + c] << (8 * e);
      }
      *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int e = max(0, a - s0); e < min(16, b - s0); ++e) at[e] = codes[(s0 - a + e) * d + c];
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
  }
  const dim3 grid((unsigned)slots, (unsigned)p.h_kv, 2);
  // a page's new tokens at most: what of it passes through LDS
  const bool one = !p.cu_seqlens && p.uniform == 1;
  const size_t lds = (size_t)(one ? 1 : p.page) * p.d;
  if (one) hipLaunchKernelGGL((cache_store_kernel<T, 64>), grid, dim3(64), lds, stream, p);
  else hipLaunchKernelGGL((cache_store_kernel<T, 256>), grid, dim3(256), lds, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_store(const CacheStoreParams& p, int dtype, hipStream_t stream) {
  if (p.tokens == 0) return hipSuccess;
  return dtype == 1 ? launch<__bf16>(p, stream) : launch<float>(p, stream);
}

}  // namespace gdn
