// gdn_cache_attention kernels: attention of each sequence's newest tokens over
// its pages of an e4m3 cache (gdn_cache_store).
//
//   s_j = scale kscale_j (q . kcode_j),  p_j = exp(s_j - max),  o = sum p_j vscale_j vcode_j / sum p_j
// The rows of one KV head are the (token, query head) pairs that share it, 16
// of them a tile: one read of the keys and values serves every query head of
// the group.  A wave takes 64 cached tokens at a time:
//   S^T = K Q^T   16x16x32 MFMA, keys as the left operand: a lane then holds
//                 the scores of ONE row for 16 tokens,
//   O^T += V^T P^T  the same lane's 16 probabilities are, as they stand, its
//                 part of the right operand: no shuffle and no LDS between the
//                 two products.
// Which token is which row of the left operand is free, so the keys' rows are
// dealt such that a lane's 16 scores belong to 16 neighbouring tokens: those
// lie in one page (pages are multiples of 16), have one scale of each kind,
// and their values are one 16-byte load from a [d][token] page.
//
// Numbers.  e4m3 codes are exact in bf16 and in fp16.  q . k runs in bf16 with
// q as it came; the probabilities, at most 1, run in fp16 (2^-12 rounding, so
// the output's own rounding is what is left).  fp32 queries and probabilities
// are split into three bf16 terms each, exact to 24 bits, and take three
// products.  Scores, maxima, sums and outputs are fp32.  The running maximum
// is that of s_j + log2 vscale_j: what multiplies the codes is then at most 1
// whatever the pages' scales are.
//
// Masks.  Scores outside a row's keys are replaced, never added to; tokens
// behind the context are cleared from the values' operand, since a code left
// there may be NaN and 0 * NaN is NaN.  A NaN among the values that some rows
// of a tile see and others do not is taken out of the product and given to
// the rows that see it (see below).  A row without keys gives zeros, and
// -inf as its logarithm of the sum.
//
// Bound by the bytes of the cache for single tokens: a wave keeps 16 to 32 KiB
// of loads in flight, straight from memory to registers (nothing is shared
// between waves, so LDS would only add a trip).  Long contexts are cut into
// pieces of equal length for enough workgroups; a second kernel joins the
// pieces by their maxima and sums, in order.
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 16;   // rows of a tile
constexpr int kTok = 64;    // tokens a wave takes at a time
constexpr int kWaves = 4;

// Eight e4m3 codes as an MFMA operand.
__device__ __forceinline__ bf16x8 to_bf16x8(uint32_t lo, uint32_t hi) {
  bf16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true),
                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true)};
  return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ f16x8 to_f16x8(uint32_t lo, uint32_t hi) {
  f16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true),
                __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true)};
  return __builtin_bit_cast(f16x8, v);
}

// f as three bf16 terms: f = a + b + c to 24 bits.
__device__ __forceinline__ void split3(const float (&f)[8], bf16x8 (&out)[3]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __bf16 a = (__bf16)f[i];
    const float r = f[i] - (float)a;
    const __bf16 b = (__bf16)r;
    out[0][i] = a;
    out[1][i] = b;
    out[2][i] = (__bf16)(r - (float)b);
  }
}
// Infinities have no remainder.
__device__ __forceinline__ void split3_any(const float (&f)[8], bf16x8 (&out)[3]) {
  split3(f, out);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (!(fabsf((float)out[0][i]) < __builtin_inff())) out[1][i] = out[2][i] = (__bf16)0.f;
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// The probabilities' operand and the values' type that goes with it.
template <typename T> struct Probs;
template <> struct Probs<__bf16> {
  static constexpr int N = 1;
  typedef f16x8 vec;
  static __device__ __forceinline__ void make(const float (&w)[8], vec (&out)[N]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[0][i] = (_Float16)w[i];
  }
  static __device__ __forceinline__ vec codes(uint32_t lo, uint32_t hi) { return to_f16x8(lo, hi); }
};
template <> struct Probs<float> {
  static constexpr int N = 3;
  typedef bf16x8 vec;
  static __device__ __forceinline__ void make(const float (&w)[8], vec (&out)[N]) { split3(w, out); }
  static __device__ __forceinline__ vec codes(uint32_t lo, uint32_t hi) { return to_bf16x8(lo, hi); }
};

// A tile of rows: its sequence, its rows' first place, and the keys any of them sees.
struct Tile {
  int n;           // sequence
  int first;       // its rows first .. first + kRows - 1 of `rows`
  int rows;        // tokens * group
  int64_t begin;   // first token
  int len;         // new tokens
  int ctx;         // tokens in the cache, the new ones among them
  int lo, hi;      // keys, lo a multiple of kTok
  bool some;       // whether there is such a tile
};

__device__ __forceinline__ Tile find_tile(const AttendParams& p, int slot, int group, int tile_rows) {
  Tile t;
  int j;
  if (!p.cu_seqlens) {
    t.n = slot / p.uniform_tiles;
    j = slot - t.n * p.uniform_tiles;
    t.begin = (int64_t)t.n * p.uniform;
    t.len = (int)p.uniform;
  } else {
    // sequence n has the slots from cu[n] group / tile_rows + n on: at least as many as its tiles
    cint32* cu = as_const(p.cu_seqlens);
    int lo = 0, hi = p.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)cu[mid] * group / tile_rows + mid <= slot) lo = mid; else hi = mid - 1;
    }
    t.n = lo;
    j = slot - (int)((int64_t)cu[lo] * group / tile_rows + lo);
    t.begin = max(cu[lo], 0);
    t.len = (int)(min((int64_t)cu[lo + 1], p.tokens) - t.begin);
  }
  t.rows = t.len * group;
  t.first = j * tile_rows;
  t.some = t.len > 0 && j >= 0 && t.first < t.rows;
  t.ctx = min(as_const(p.lens)[t.n], p.max_tokens);  // contexts end with the table
  if (!t.some) return t;
  const int t0 = t.first / group, t1 = min(t.len - 1, (t.first + tile_rows - 1) / group);
  t.hi = p.causal ? min(t.ctx, t.ctx - t.len + t1 + 1) : t.ctx;
  t.lo = p.window ? max(0, t.ctx - t.len + t0 - p.window + 1) : 0;
  t.lo &= ~(kTok - 1);
  if (t.hi < t.lo) t.hi = t.lo;
  return t;
}

__device__ __forceinline__ int pieces(const AttendParams& p, const Tile& t) {
  return max(1, (t.hi - t.lo + p.piece - 1) / p.piece);
}

// A byte mask of the codes among four that are NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t m = ((w & 0x7f7f7f7fu) ^ 0x7f7f7f7fu) + 0x7f7f7f7fu;  // bit 7 of a byte set unless its code is NaN
  return (~m & 0x80808080u) >> 7;                                      // 1 where NaN
}

template <typename T>
__device__ __forceinline__ float gated(const AttendParams& p, float o, int64_t token, int64_t at) {
  if (!p.gate) return o;
  const float z = to_f32(reinterpret_cast<const T*>(p.gate)[token * p.gate_stride + at]);
  return o / (1.f + (sizeof(T) == 2 ? __expf(-z) : expf(-z)));
}

template <typename T, int D>
__global__ __launch_bounds__(kWaves * 64, 2) void attend_kernel(AttendParams p) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int NQ = F32 ? 3 : 1;
  constexpr int KS = D / 32, MT = D / 16;
  typedef Probs<T> P;
  __shared__ float s_o[kWaves][kRows][D + 4];
  __shared__ float s_m[kWaves][kRows], s_l[kWaves][kRows];

  const int group = p.h_q / p.h_kv;
  const int head = blockIdx.y, piece = blockIdx.z;
  const Tile tile = find_tile(p, blockIdx.x, group, kRows);
  if (!tile.some) return;
  const int ns = pieces(p, tile);
  if (piece >= ns) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;

  // this lane's row
  const int row = tile.first + r;
  const bool live = row < tile.rows;  // the last tile's other rows see nothing and are not written
  const int tok = row / group, hq = head * group + (row - tok * group);
  const int pos = tile.ctx - tile.len + tok;
  const int row_hi = live ? (p.causal ? min(tile.ctx, pos + 1) : tile.ctx) : 0;
  const int row_lo = p.window ? pos - p.window + 1 : 0;

  // Q: lane (row r, group g) holds elements 64 b + 16 g .. + 15 of each 64, the order its keys come in
  bf16x8 q[KS][NQ];
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const int at = (k / 2) * 64 + g * 16 + (k & 1) * 8;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) load8(reinterpret_cast<const T*>(p.q) + (tile.begin + tok) * p.q_stride + (int64_t)hq * D + at, f);
    if constexpr (F32) {
      split3_any(f, q[k]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[k][0][i] = (__bf16)f[i];
    }
  }

  f32x4 o[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -__builtin_inff(), l = 0.f;

  const int start = tile.lo + piece * p.piece;
  const int stop = min(tile.hi, start + p.piece);
  const int32_t* table = p.page_table + (int64_t)tile.n * p.max_pages;
  const int page = 1 << p.page_shift, in_page = page - 1;
  const int kg = r >> 2, ki = r & 3;  // this lane's row of the keys' operand: token 16 kg + 4 tt + ki
  for (int k0 = start + wave * kTok; k0 < stop; k0 += kWaves * kTok) {
    // pages of this lane's 16 tokens as a row of the keys, and as a column of the scores
    const int tk = k0 + 16 * kg, ts = k0 + 16 * g;
    int pk = tk < stop ? table[tk >> p.page_shift] : -1;
    int ps = ts < stop ? table[ts >> p.page_shift] : -1;
    const bool held = ps >= 0 && ps < p.pages;  // a page outside the pool holds nothing
    pk = pk >= 0 && pk < p.pages ? pk : 0;
    ps = held ? ps : 0;
    const float ks = p.k_scale[(int64_t)ps * p.h_kv + head], vs = p.v_scale[(int64_t)ps * p.h_kv + head];
    const uint8_t* kp = p.k_cache + ((((int64_t)pk * p.h_kv + head) << p.page_shift) + (tk & in_page) + ki) * D + g * 16;
    const uint8_t* vp = p.v_cache + ((((int64_t)ps * p.h_kv + head) * D) << p.page_shift) + (ts & in_page);
    uint4 kc[4][D / 64], vc[MT];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt)
#pragma unroll
      for (int b = 0; b < D / 64; ++b) kc[tt][b] = *reinterpret_cast<const uint4*>(kp + tt * 4 * D + b * 64);
#pragma unroll
    for (int i = 0; i < MT; ++i) vc[i] = *reinterpret_cast<const uint4*>(vp + ((i * 16 + r) << p.page_shift));

    f32x4 s[4];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) s[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const bf16x8 k_lo = to_bf16x8(kc[tt][b].x, kc[tt][b].y), k_hi = to_bf16x8(kc[tt][b].z, kc[tt][b].w);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          s[tt] = mfma(k_lo, q[2 * b][NQ - 1 - i], s[tt]);
          s[tt] = mfma(k_hi, q[2 * b + 1][NQ - 1 - i], s[tt]);
        }
      }

    // this lane's row against tokens ts .. ts + 15 (s[tt][i]: token ts + 4 tt + i): it sees from .. to - 1 of them
    const float f = ks * p.scale_log2;
    const int from = max(0, min(row_lo - ts, 16)), to = held ? max(0, min(row_hi - ts, 16)) : 0;
    const bool sees = from < to;
    const bool part = __any(live && (from > 0 || to < 16));  // some row sees some of the tile only
    if (part) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (e < from || e >= to) s[e >> 2][e & 3] = -__builtin_inff();
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, s[e >> 2][e & 3]);
    // (the scales are positive, so the largest product is that of the largest score)
    top = sees ? fmaf(top, f, fminf(fmaxf(__log2f(fabsf(vs)), -40.f), 120.f)) : -__builtin_inff();
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float now = fmaxf(m, top);
    const float base = now == -__builtin_inff() ? 0.f : now;
    const float alpha = __builtin_amdgcn_exp2f(m - base);
    m = now;
    float w[2][8], sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e >> 3][e & 7] = __builtin_amdgcn_exp2f(fmaf(s[e >> 2][e & 3], f, -base));
    if (part) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (e < from || e >= to) w[e >> 3][e & 7] = 0.f;
    }
    const float factor = sees ? vs : 0.f;  // whatever stands where no page is
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      sum += w[e >> 3][e & 7];
      w[e >> 3][e & 7] *= factor;
    }
    l = l * alpha + sum;

    if (part) {
      // codes that must not reach the product: tokens behind the context, or of no page
      const int keep = held ? max(0, min(tile.ctx - ts, 16)) : 0;
      uint32_t mask[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = keep - 4 * i;
        mask[i] = k >= 4 ? 0xffffffffu : k <= 0 ? 0u : (1u << (8 * k)) - 1;
      }
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        vc[i].x &= mask[0]; vc[i].y &= mask[1]; vc[i].z &= mask[2]; vc[i].w &= mask[3];
        bad |= nan_bytes(vc[i].x) | nan_bytes(vc[i].y) | nan_bytes(vc[i].z) | nan_bytes(vc[i].w);
      }
      if (__any(bad != 0)) {
        // NaN codes leave the product; rows that see one get NaN there, by a product of
        // ones (a code is NaN) and ones (a row sees the token)
        float one[2][8];
#pragma unroll
        for (int e = 0; e < 16; ++e) one[e >> 3][e & 7] = e >= from && e < to ? 1.f : 0.f;
        typename P::vec see[2][P::N];
        P::make(one[0], see[0]);
        P::make(one[1], see[1]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint4 c = vc[i];
          const uint4 nn = make_uint4(nan_bytes(c.x), nan_bytes(c.y), nan_bytes(c.z), nan_bytes(c.w));
          f32x4 hit = f32x4{0.f, 0.f, 0.f, 0.f};
          hit = mfma(P::codes(nn.x * 0x38u, nn.y * 0x38u), see[0][0], hit);  // 0x38: 1.0
          hit = mfma(P::codes(nn.z * 0x38u, nn.w * 0x38u), see[1][0], hit);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] = hit[e] > 0.f ? __builtin_nanf("") : o[i][e];
          vc[i] = make_uint4(c.x & ~(nn.x * 0xffu), c.y & ~(nn.y * 0xffu), c.z & ~(nn.z * 0xffu), c.w & ~(nn.w * 0xffu));
        }
      }
    }
    typename P::vec pw[2][P::N];
    P::make(w[0], pw[0]);
    P::make(w[1], pw[1]);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      o[i] *= alpha;
      const typename P::vec v_lo = P::codes(vc[i].x, vc[i].y), v_hi = P::codes(vc[i].z, vc[i].w);
#pragma unroll
      for (int e = 0; e < P::N; ++e) {
        o[i] = mfma(v_lo, pw[0][P::N - 1 - e], o[i]);
        o[i] = mfma(v_hi, pw[1][P::N - 1 - e], o[i]);
      }
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // join the waves
  if (g == 0) s_m[wave][r] = m, s_l[wave][r] = l;
#pragma unroll
  for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(&s_o[wave][r][i * 16 + g * 4]) = o[i];
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * D / 4; i += kWaves * 64) {
    const int rr = i / (D / 4), c = (i - rr * (D / 4)) * 4, at = tile.first + rr;
    if (at >= tile.rows) break;
    float mm = s_m[0][rr];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) mm = fmaxf(mm, s_m[k][rr]);
    const float base = mm == -__builtin_inff() ? 0.f : mm;
    f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
    float ll = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      const float a = __builtin_amdgcn_exp2f(s_m[k][rr] - base);
      ll += a * s_l[k][rr];
      sum += a * *reinterpret_cast<const f32x4*>(&s_o[k][rr][c]);
    }
    const int64_t token = tile.begin + at / group;
    const int h = head * group + at % group;
    const int64_t out = token * p.h_q + h;
    if (ns == 1) {
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = gated<T>(p, sum[e] * inv, token, (int64_t)h * D + c + e);
      store4(reinterpret_cast<T*>(p.o) + token * p.o_stride + (int64_t)h * D + c, y);
      if (p.lse && c == 0) p.lse[out] = ll == 0.f ? -__builtin_inff() : (mm + __log2f(ll)) * 0.69314718055994530942f;
    } else {
      const int64_t part = (int64_t)piece * p.tokens * p.h_q + out;
      *reinterpret_cast<f32x4*>(p.part_o + part * D + c) = sum;
      if (c == 0) p.part_ml[2 * part] = mm, p.part_ml[2 * part + 1] = ll;
    }
  }
}

// Joins the pieces of a row: a wave a row, its lanes over the head's elements.
template <typename T, int D>
__global__ __launch_bounds__(256) void join_kernel(AttendParams p) {
  const int group = p.h_q / p.h_kv, lane = threadIdx.x & 63;
  const Tile tile = find_tile(p, blockIdx.x, group, kRows);
  if (!tile.some) return;
  const int ns = pieces(p, tile);
  if (ns == 1) return;  // written already
  for (int rr = threadIdx.x >> 6; rr < kRows; rr += 4) {
    const int at = tile.first + rr;
    if (at >= tile.rows) return;
    const int64_t token = tile.begin + at / group;
    const int h = blockIdx.y * group + at % group;
    const int64_t out = token * p.h_q + h, step = p.tokens * p.h_q;
    float mm = -__builtin_inff();
    for (int s = 0; s < ns; ++s) mm = fmaxf(mm, p.part_ml[2 * (s * step + out)]);
    const float base = mm == -__builtin_inff() ? 0.f : mm;
    constexpr int E = D / 64;
    float sum[E], ll = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = 0.f;
    for (int s = 0; s < ns; ++s) {
      const int64_t part = s * step + out;
      const float a = __builtin_amdgcn_exp2f(p.part_ml[2 * part] - base);
      ll += a * p.part_ml[2 * part + 1];
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += a * p.part_o[part * D + e * 64 + lane];
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t c = (int64_t)h * D + e * 64 + lane;
      reinterpret_cast<T*>(p.o)[token * p.o_stride + c] = from_f32<T>(gated<T>(p, sum[e] * inv, token, c));
    }
    if (p.lse && lane == 0) p.lse[out] = ll == 0.f ? -__builtin_inff() : (mm + __log2f(ll)) * 0.69314718055994530942f;
  }
}

// How a call is cut: tiles of rows, and pieces of the context of `piece` tokens.
struct Plan {
  int64_t slots;  // tiles at most
  int32_t uniform_tiles;
  int64_t uniform;
  int32_t piece;
  int64_t pieces;  // of the longest context that the table holds
};

// Tokens that a row of the page table holds; positions are 32-bit.
int32_t max_tokens(const AttendShape& a) {
  const int64_t most = (int64_t)a.max_pages * a.page;
  return (int32_t)(most < (1 << 30) ? most : (1 << 30));
}

Plan plan(const AttendShape& a) {
  Plan c;
  const int64_t group = a.h_q / a.h_kv;
  c.uniform = a.tokens / a.n_seqs;
  c.uniform_tiles = (int32_t)((c.uniform * group + kRows - 1) / kRows);
  c.slots = a.ragged ? a.tokens * group / kRows + a.n_seqs : (int64_t)c.uniform_tiles * a.n_seqs;
  // Pieces: about 4096 workgroups where the contexts allow it (16 for each CU: unequal contexts then even
  // out), of at least 256 tokens, a turn of a workgroup's four waves.
  const int64_t most = max_tokens(a), step = kWaves * kTok;
  const double even = (double)most * a.h_kv * c.slots / 4096;
  int64_t piece = even >= (double)most ? most : (int64_t)even;
  piece = (piece + step - 1) / step * step;
  c.piece = (int32_t)(piece < step ? step : piece);
  c.pieces = (most + c.piece - 1) / c.piece;
  if (c.pieces < 1) c.pieces = 1;
  return c;
}

template <typename T, int D>
hipError_t launch(AttendParams p, const Plan& c, hipStream_t stream) {
  hipLaunchKernelGGL((attend_kernel<T, D>), dim3((unsigned)c.slots, (unsigned)p.h_kv, (unsigned)c.pieces), dim3(kWaves * 64), 0,
                     stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || c.pieces == 1) return e;
  hipLaunchKernelGGL((join_kernel<T, D>), dim3((unsigned)c.slots, (unsigned)p.h_kv), dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_d(const AttendParams& p, const Plan& c, int d, hipStream_t stream) {
  switch (d) {
    case 64: return launch<T, 64>(p, c, stream);
    case 128: return launch<T, 128>(p, c, stream);
    default: return launch<T, 256>(p, c, stream);
  }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t attend_workspace_bytes(const AttendShape& a) {
  if (a.tokens == 0) return 0;
  const Plan c = plan(a);
  if (c.pieces == 1) return 0;
  const size_t rows = (size_t)c.pieces * a.tokens * a.h_q;
  return round256(rows * a.d * sizeof(float)) + round256(rows * 2 * sizeof(float));
}

hipError_t launch_attend(AttendParams p, const AttendShape& a, void* workspace, int dtype, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  const Plan c = plan(a);
  p.max_tokens = max_tokens(a);
  p.uniform = c.uniform;
  p.uniform_tiles = c.uniform_tiles;
  p.piece = c.piece;
  if (c.pieces > 1) {
    const size_t rows = (size_t)c.pieces * a.tokens * a.h_q;
    p.part_o = reinterpret_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + round256(rows * a.d * sizeof(float)));
  }
  return dtype == 1 ? launch_d<__bf16>(p, c, a.d, stream) : launch_d<float>(p, c, a.d, stream);
}

}  // namespace gdn
