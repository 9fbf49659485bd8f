// gdn_rms_norm and gdn_rms_norm_backward kernels: RMS norm of rows, fused with
// the residual sum ahead of it (or the residual sum after it), the residual
// scale and the output gate.
//
//   pre :  h = residual + s x,  y = h r (w + c) act(z)          (y and h out)
//   post:  y = residual + s x r (w + c) act(z)
//   r = (mean(h^2) + eps)^-1/2 over the row (of x in the post order)
//
// Both directions are bound by the bytes they move: a row is read once into
// registers by a group of lanes, reduced once, and written once.  The group is
// as small as the row allows (16 lanes for a head of 128 in bf16, a wave up to
// 1,024 elements, a workgroup beyond), so that short rows keep every lane busy
// and need no LDS.  16384 rows of 5120 with a residual: 127 us, 5.3 TB/s read and
// written, where a large copy reaches 5.1; one row: 5.5 us, a launch.  Statistics, products and sums are fp32; the only rounding
// to the io dtype is each output's.  y of the pre order is formed from the
// unrounded h.
//
// Backward, with n = h r, u = dy' (w + c) act(z), dy' = s dy in the post order:
//   dh = r (u - n mean(u n)) + d_sum,   dz = dy' n (w + c) act'(z),
//   dw = sum over rows of dy' n act(z).
// mean(u n) = r mean(u h): both row sums (h^2 and u h) are taken in one pass.
// dw: a group adds its rows in registers, the groups of a workgroup join in
// LDS, each workgroup leaves one partial row, and a second kernel adds the
// partial rows in order: the result does not depend on timing.  8192 tokens of
// 32 heads of 128 with a gate: 79 us, 4.3 TB/s (147 before the weights
// and the next row were read wide and ahead of the present row's sums).
#include "gdn_device.h"
#include "gdn_internal.h"

#include <type_traits>

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC > 16 ? 16 : sizeof(T) * VEC) Pack {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const void* base, int64_t at) {
  return *reinterpret_cast<const Pack<T, VEC>*>(reinterpret_cast<const T*>(base) + at);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(void* base, int64_t at, const float (&f)[VEC]) {
  Pack<T, VEC> p;
#pragma unroll
  for (int e = 0; e < VEC; ++e) p.v[e] = from_f32<T>(f[e]);
  *reinterpret_cast<Pack<T, VEC>*>(reinterpret_cast<T*>(base) + at) = p;
}

// Weights are bf16 or fp32 whatever the rows are; without any they are ones.
template <int VEC>
struct Weight {
  Pack<float, VEC> v;  // fp32 as it is, bf16 in its first half
  __device__ __forceinline__ void load(const void* w, int bf16, int at) {
    if (!w) return;
    if (bf16) {
      const Pack<__bf16, VEC> h = load_pack<__bf16, VEC>(w, at);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v.v[e] = to_f32(h.v[e]);
    } else {
      v = load_pack<float, VEC>(w, at);
    }
  }
  __device__ __forceinline__ float get(const void* w, float offset, int e) const { return w ? offset + v.v[e] : 1.0f; }
};

// Sigmoid: the hardware exponential for bf16 rows; for fp32 rows expf, whose
// error stays at an ulp for large arguments.
template <typename T>
__device__ __forceinline__ float sigmoid(float z);
template <>
__device__ __forceinline__ float sigmoid<__bf16>(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }
template <>
__device__ __forceinline__ float sigmoid<float>(float z) { return 1.0f / (1.0f + expf(-z)); }

// Sums of N values over a group of G lanes; every lane receives them.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&a)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = G == 16 ? row16_sum(a[i]) : wave_sum(a[i]);
  if constexpr (G == kThreads) {
    __shared__ float s[N][kThreads / 64];
    __syncthreads();  // the previous row's sums have been read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i][threadIdx.x >> 6] = a[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = (s[i][0] + s[i][1]) + (s[i][2] + s[i][3]);
  }
}

template <typename T, int VEC, int G, int NV>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormParams p) {
  const int lane = threadIdx.x % G;
  int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kThreads / G) + threadIdx.x / G;
  const bool live = row < p.rows;
  if (!live) row = p.rows - 1;  // a surplus group follows along without storing
  const uint32_t t = (uint32_t)row / (uint32_t)p.heads;
  const int64_t col = (int64_t)((uint32_t)row - t * (uint32_t)p.heads) * p.width;
  const bool sum = p.order == 0 && p.residual;

  Pack<T, VEC> x[NV], res[NV], z[NV];
  Weight<VEC> w[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = (v * G + lane) * VEC;
    if (at >= p.width) continue;
    x[v] = load_pack<T, VEC>(p.x, t * p.x_stride + col + at);
    if (p.residual) res[v] = load_pack<T, VEC>(p.residual, t * p.residual_stride + col + at);
    if (p.gate) z[v] = load_pack<T, VEC>(p.gate, t * p.gate_stride + col + at);
    w[v].load(p.weight, p.weight_bf16, at);
  }
  float h[NV][VEC], ss[1] = {0.f};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if ((v * G + lane) * VEC >= p.width) continue;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      h[v][e] = to_f32(x[v].v[e]);
      if (sum) h[v][e] = fmaf(p.scale, h[v][e], to_f32(res[v].v[e]));
      ss[0] = fmaf(h[v][e], h[v][e], ss[0]);
    }
  }
  group_sum<G>(ss);
  const float r = 1.0f / sqrtf(ss[0] / (float)p.width + p.eps);
  if (!live) return;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = (v * G + lane) * VEC;
    if (at >= p.width) continue;
    float y[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      y[e] = h[v][e] * r * w[v].get(p.weight, p.weight_offset, e);
      if (p.gate) {
        const float zz = to_f32(z[v].v[e]), s = sigmoid<T>(zz);
        y[e] *= p.act == 1 ? zz * s : s;
      }
      if (p.order == 1) y[e] = p.residual ? fmaf(p.scale, y[e], to_f32(res[v].v[e])) : p.scale * y[e];
    }
    if (sum) store_pack<T, VEC>(p.sum, t * p.sum_stride + col + at, h[v]);
    store_pack<T, VEC>(p.y, t * p.y_stride + col + at, y);
  }
}

// GATE: without one a wide row leaves registers for another workgroup (16384 rows of 5120: 275 -> 186 us; of 8192:
// 387 -> 216).
template <typename T, int VEC, int G, int NV, bool GATE>
__global__ __launch_bounds__(kThreads, NV * VEC > 16 && NV * VEC <= 32 ? 2 : 1) void norm_backward_kernel(NormBwdParams p, float* partial) {
  constexpr int kGroups = kThreads / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const bool gate = GATE && (NV > 2 || p.gate);  // (the test costs nothing and leaves short rows their registers: 124, 136 without)
  float dw[NV][VEC];
  Weight<VEC> w[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = (v * G + lane) * VEC;
    if (at < p.width) w[v].load(p.weight, p.weight_bf16, at);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[v][e] = 0.f;
  }

  struct Row {
    Pack<T, VEC> x[NV], g[NV], z[NV], ds[NV];
  };
  // every group of a workgroup makes the same number of turns; one beyond the last row follows along on that row
  auto at_row = [&](int64_t row, uint32_t& t, int64_t& col) {
    const uint32_t r = (uint32_t)(row < p.rows ? row : p.rows - 1);
    t = r / (uint32_t)p.heads;
    col = (int64_t)(r - t * (uint32_t)p.heads) * p.width;
  };
  auto load = [&](Row& d, int64_t row) {
    uint32_t t;
    int64_t col;
    at_row(row, t, col);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (v * G + lane) * VEC;
      if (at >= p.width) continue;
      d.x[v] = load_pack<T, VEC>(p.x, t * p.x_stride + col + at);
      d.g[v] = load_pack<T, VEC>(p.dy, t * p.dy_stride + col + at);
      if (gate) d.z[v] = load_pack<T, VEC>(p.gate, t * p.gate_stride + col + at);
      if (p.d_sum) d.ds[v] = load_pack<T, VEC>(p.d_sum, t * p.d_sum_stride + col + at);
    }
  };
  const float post = p.order == 1 ? p.scale : 1.0f, inv_width = 1.0f / (float)p.width;
  auto work = [&](const Row& d, int64_t row) {
    float sums[2] = {0.f, 0.f};  // of h^2 and of u h
    float s[NV][VEC];            // sigmoid of the gate
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if ((v * G + lane) * VEC >= p.width) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float h = to_f32(d.x[v].v[e]);
        float u = to_f32(d.g[v].v[e]) * w[v].get(p.weight, p.weight_offset, e);
        if (gate) {
          const float z = to_f32(d.z[v].v[e]);
          s[v][e] = sigmoid<T>(z);
          u *= p.act == 1 ? z * s[v][e] : s[v][e];
        }
        sums[0] = fmaf(h, h, sums[0]);
        sums[1] = fmaf(u, h, sums[1]);
      }
    }
    group_sum<G>(sums);
    const float r = 1.0f / sqrtf(sums[0] * inv_width + p.eps);
    const float mean = post * r * (sums[1] * inv_width);  // of u n
    if (row >= p.rows) return;
    uint32_t t;
    int64_t col;
    at_row(row, t, col);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (v * G + lane) * VEC;
      if (at >= p.width) continue;
      float dx[VEC], dz[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float n = to_f32(d.x[v].v[e]) * r, dy = post * to_f32(d.g[v].v[e]), wt = w[v].get(p.weight, p.weight_offset, e);
        float a = 1.f;
        const float nd = dy * n;
        if (gate) {
          const float z = to_f32(d.z[v].v[e]), sg = s[v][e];
          a = p.act == 1 ? z * sg : sg;
          dz[e] = nd * wt * (p.act == 1 ? sg * (1.f + z * (1.f - sg)) : sg * (1.f - sg));
        }
        dx[e] = r * fmaf(-n, mean, dy * wt * a);
        if (p.d_sum) dx[e] += to_f32(d.ds[v].v[e]);
        dw[v][e] = fmaf(nd, a, dw[v][e]);
      }
      if (p.d_residual) store_pack<T, VEC>(p.d_residual, t * p.d_residual_stride + col + at, dx);
      if (p.dx) {
        if (p.order == 0)
#pragma unroll
          for (int e = 0; e < VEC; ++e) dx[e] *= p.scale;
        store_pack<T, VEC>(p.dx, t * p.dx_stride + col + at, dx);
      }
      if (gate) store_pack<T, VEC>(p.dgate, t * p.dgate_stride + col + at, dz);
    }
  };

  const int64_t step = (int64_t)gridDim.x * kGroups;
  const int64_t begin = (int64_t)blockIdx.x * kGroups;
  if constexpr (NV * VEC <= 24) {
    // the next row is on its way while one is worked on (it is no row's output: p.dx and the others may be an
    // input's own rows, but each row is read by the group that writes it)
    Row a, b;
    if (begin < p.rows) load(a, begin + group);
    for (int64_t first = begin; first < p.rows; first += 2 * step) {
      const bool second = first + step < p.rows;
      if (second) load(b, first + step + group);
      work(a, first + group);
      if (!second) break;
      if (first + 2 * step < p.rows) load(a, first + 2 * step + group);
      work(b, first + step + group);
    }
  } else {
    for (int64_t first = begin; first < p.rows; first += step) {
      Row a;
      load(a, first + group);
      work(a, first + group);
    }
  }
  if (!partial) return;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (v * G + lane) * VEC;
      if (at >= p.width) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) partial[(int64_t)blockIdx.x * p.width + at + e] = dw[v][e];
    }
  } else {
    __shared__ float s[kGroups][G * NV * VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[group][(v * G + lane) * VEC + e] = dw[v][e];
    __syncthreads();
    for (int at = threadIdx.x; at < p.width; at += kThreads) {
      float a = 0.f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) a += s[k][at];
      partial[(int64_t)blockIdx.x * p.width + at] = a;
    }
  }
}

// dw[c] = sum of the partial rows: 16 columns a workgroup, 64 row lanes, four rows of each at a time; the lanes'
// sums join in LDS in a fixed order.
__global__ __launch_bounds__(1024) void norm_dweight_kernel(const float* partial, int blocks, int width, float* dw) {
  __shared__ float s[64][17];
  const int c = threadIdx.x & 15, k = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  if (col < width)
    for (int b = k; b < blocks; b += 256)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (b + 64 * i < blocks) a[i] += partial[(int64_t)(b + 64 * i) * width + col];
  s[k][c] = (a[0] + a[1]) + (a[2] + a[3]);
  __syncthreads();
  if (k < 8) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += s[k * 8 + i][c];
    s[k * 8][c] = t;
  }
  __syncthreads();
  if (k == 0 && col < width) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += s[i * 8][c];
    dw[col] = t;
  }
}

bool vec_ok(const void* p, int64_t stride, int vec, size_t es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (vec * es) == 0 && stride % vec == 0);
}

// Calls f with the template arguments that fit a row: VEC elements a load,
// groups of G lanes, NV loads a lane.  `vec`: whether 16-byte loads are aligned.
// Heads of 128 with a wave each instead of 16 lanes: 231 us backward, 82 with;
// rows of 512 with a workgroup instead of a wave: 198 and 110, of 1024: 128 and
// 120.
template <typename T, typename F>
hipError_t dispatch(int width, bool vec, F&& f) {
  constexpr int V = 16 / (int)sizeof(T);
  auto with = [&](auto ve, auto g, auto nv) { return f.template operator()<decltype(ve)::value, decltype(g)::value, decltype(nv)::value>(); };
#define GDN_NORM(VE, G, NV) \
  return with(std::integral_constant<int, VE>{}, std::integral_constant<int, G>{}, std::integral_constant<int, NV>{})
  if (vec && width % V == 0) {
    const int n = width / V;
    if (n <= 16) GDN_NORM(V, 16, 1);
    if (n <= 64) GDN_NORM(V, 64, 1);
    if (n <= 128) GDN_NORM(V, 64, 2);
    const int per = (n + 255) / 256;
    if (per <= 1) GDN_NORM(V, 256, 1);
    if (per <= 2) GDN_NORM(V, 256, 2);
    if (per <= 3) GDN_NORM(V, 256, 3);
    if (per <= 4) GDN_NORM(V, 256, 4);
    if (per <= 6) GDN_NORM(V, 256, 6);
    if (per <= 8) GDN_NORM(V, 256, 8);
    if constexpr (V == 4) GDN_NORM(V, 256, 16);
  }
  if (width <= 16) GDN_NORM(1, 16, 1);
  if (width <= 128) GDN_NORM(1, 64, 2);
  if (width <= 512) GDN_NORM(1, 64, 8);
  if (width <= 2048) GDN_NORM(1, 256, 8);
  if (width <= 4096) GDN_NORM(1, 256, 16);  // 7095 rows of 3559 with a gate: 83 us, 118 with 24 loads
  if (width <= 6144) GDN_NORM(1, 256, 24);
  GDN_NORM(1, 256, 64);
#undef GDN_NORM
}

// The most workgroups of the backward: enough to fill the chip, few enough
// that their partial dw rows stay small beside the rows themselves (8192 tokens
// of 32 gated heads of 128: 82 us, 90 with 512, 86 with 2048).
constexpr int kMostBlocks = 1024;
int backward_blocks(int64_t rows) {
  return (int)(rows < kMostBlocks ? (rows > 0 ? rows : 1) : kMostBlocks);
}

template <typename T>
struct Forward {
  const NormParams& p;
  hipStream_t stream;
  template <int VEC, int G, int NV>
  hipError_t operator()() const {
    // a grid's first side holds less than 2^32 threads: 2^22 workgroups, and as many sides as it takes
    const int64_t per = kThreads / G, need = (p.rows + per - 1) / per, side = need < (1 << 22) ? need : 1 << 22;
    hipLaunchKernelGGL((norm_kernel<T, VEC, G, NV>), dim3((unsigned)side, (unsigned)((need + side - 1) / side)), dim3(kThreads),
                       0, stream, p);
    return hipGetLastError();
  }
};
template <typename T>
struct Backward {
  const NormBwdParams& p;
  hipStream_t stream;
  int* blocks;  // in: the most; out: the number launched
  template <int VEC, int G, int NV>
  hipError_t operator()() const {
    const int64_t need = (p.rows + kThreads / G - 1) / (kThreads / G);
    // as many as run at once, or a whole number of times that: three of these run on a CU (65536 rows of 1024 without
    // a gate: 131 us with 1024, 103 with 768), two or four of the others
    if (sizeof(T) == 2 && G > 16 && NV <= 2 && VEC > 1 && !p.gate && *blocks > 768) *blocks = 768;
    if (need < *blocks) *blocks = (int)need;
    if (p.dweight && need == 2) *blocks = 1;  // two turns of one workgroup take less time than a second launch (10 -> 7.5 us)
    float* partial = !p.dweight ? nullptr : *blocks == 1 ? p.dweight : reinterpret_cast<float*>(p.workspace);
    if (p.gate) hipLaunchKernelGGL((norm_backward_kernel<T, VEC, G, NV, true>), dim3((unsigned)*blocks), dim3(kThreads), 0, stream, p, partial);
    else hipLaunchKernelGGL((norm_backward_kernel<T, VEC, G, NV, false>), dim3((unsigned)*blocks), dim3(kThreads), 0, stream, p, partial);
    return hipGetLastError();
  }
};

template <typename T>
hipError_t forward(const NormParams& p, hipStream_t stream) {
  constexpr int V = 16 / (int)sizeof(T);
  const size_t es = sizeof(T);
  const bool vec = p.width % V == 0 && vec_ok(p.weight, 0, V, p.weight_bf16 ? 2 : 4) && vec_ok(p.x, p.x_stride, V, es) && vec_ok(p.gate, p.gate_stride, V, es) &&
                   vec_ok(p.residual, p.residual_stride, V, es) && vec_ok(p.y, p.y_stride, V, es) &&
                   vec_ok(p.sum, p.sum_stride, V, es);
  return dispatch<T>(p.width, vec, Forward<T>{p, stream});
}
template <typename T>
hipError_t backward(const NormBwdParams& p, hipStream_t stream, int* blocks) {
  constexpr int V = 16 / (int)sizeof(T);
  const size_t es = sizeof(T);
  const bool vec = p.width % V == 0 && vec_ok(p.weight, 0, V, p.weight_bf16 ? 2 : 4) && vec_ok(p.x, p.x_stride, V, es) && vec_ok(p.gate, p.gate_stride, V, es) &&
                   vec_ok(p.dy, p.dy_stride, V, es) && vec_ok(p.d_sum, p.d_sum_stride, V, es) &&
                   vec_ok(p.dx, p.dx_stride, V, es) && vec_ok(p.dgate, p.dgate_stride, V, es) &&
                   vec_ok(p.d_residual, p.d_residual_stride, V, es);
  return dispatch<T>(p.width, vec, Backward<T>{p, stream, blocks});
}

}  // namespace

size_t norm_backward_workspace_bytes(int64_t rows, int width) {
  return (size_t)backward_blocks(rows) * width * sizeof(float);
}

hipError_t launch_norm(const NormParams& p, int dtype, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  return dtype == 1 ? forward<__bf16>(p, stream) : forward<float>(p, stream);
}

hipError_t launch_norm_backward(const NormBwdParams& p, int dtype, hipStream_t stream) {
  int blocks = 0;  // no rows: dw is the sum of nothing
  if (p.rows > 0) {
    blocks = backward_blocks(p.rows);
    const hipError_t e = dtype == 1 ? backward<__bf16>(p, stream, &blocks) : backward<float>(p, stream, &blocks);
    if (e != hipSuccess) return e;
  }
  if (!p.dweight || blocks == 1) return hipSuccess;  // one workgroup's sums are dw
  hipLaunchKernelGGL(norm_dweight_kernel, dim3((unsigned)((p.width + 15) / 16)), dim3(1024), 0, stream,
                     reinterpret_cast<const float*>(p.workspace), blocks, p.width, p.dweight);
  return hipGetLastError();
}

}  // namespace gdn
