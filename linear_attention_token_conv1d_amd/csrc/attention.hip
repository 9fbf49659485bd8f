// gdn_cache_attention kernels: attention of each sequence's newest tokens over
// its pages of an e4m3 cache (gdn_cache_store).
//
//   s_j = scale kscale_j (q . kcode_j),  p_j = exp(s_j - max),  o = sum p_j vscale_j vcode_j / sum p_j
// The rows of one KV head are the (token, query head) pairs that share it: one
// read of the keys and values serves every query head of the group.  Two
// kernels, of 16 rows a workgroup (single and few tokens) and of 128 (chunks).
// In both a wave forms
//   S^T = K Q^T     keys as the left operand: a lane then holds the scores of
//                   ONE row for 16 tokens,
//   O^T += V^T P^T  the same lane's 16 weights are, as they stand, its part of
//                   the right operand: no shuffle and no LDS between the two
//                   products.
// Which token is which row of the left operand is free, so the keys' rows are
// dealt such that a lane's 16 scores belong to 16 neighbouring tokens: those
// lie in one page (pages are multiples of 16), have one scale of each kind,
// and their values are one 16-byte load from a [d][token] page.
//
// Numbers.  e4m3 codes are exact in bf16 and in fp16.  q . k runs in bf16 with
// q as it came; the weights p_j vscale_j, below 256, run in fp16 (2^-12
// rounding, so the output's own rounding is what is left).  fp32 queries and
// weights are split into three bf16 terms each, exact to 24 bits, and take
// three products.  Scores, maxima, sums and outputs are fp32.  The running
// maximum is that of s_j + log2 vscale_j, and moves only where it grows by
// more than 2^8: the outputs are seldom multiplied again.
//
// Masks.  Scores outside a row's keys are replaced, never added to; tokens
// behind the context are cleared from the values' operand, since a code left
// there may be NaN and 0 * NaN is NaN.  A NaN among the values that some rows
// of a tile see and others do not is taken out of the product and given to
// the rows that see it (see below).  A row without keys gives zeros, and
// -inf as its logarithm of the sum.
//
// 16 rows: a wave takes 64 tokens at a time by 16x16x32 MFMA.  Bound by the
// bytes of the cache: a wave keeps 16 to 32 KiB of loads on their way, straight
// from memory to registers (nothing is shared between waves, so LDS would only
// add a trip).  Long contexts are cut into pieces, or all work into equal
// shares; a second kernel joins the partial results by their maxima and sums,
// in order.  One token each of 64 sequences of 4096 to 32768, 4 KV heads of 256
// under 24: 364 us, 5.7 TB/s of codes, where a bare read reaches 6.2.
// 128 rows: bound by the vector instructions that run beside the matrix units
// (codes to operands, exponentials).  4096 tokens over 8097, the same heads:
// 616 us, 989 TFLOP/s, where a library product of 8192^3 in bf16 reaches 1128.
#include "gdn_device.h"
#include "gdn_internal.h"
#include "sequences.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

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

// The largest of the four lanes r, r + 16, r + 32, r + 48, for each of them.
__device__ __forceinline__ float group_max(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

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
  int all_lo, all_hi;  // keys that every row sees
  bool some;       // whether there is such a tile
};

// The keys that the tile's sequence's new token i sees: from keys_from to keys_to - 1, both in [0, ctx].  (Neither a
// position before the first key nor a window of 2^31 - 1 may pass 32 bits.)
__device__ __forceinline__ int keys_to(const AttendParams& p, const Tile& t, int i) {
  return p.causal ? max(0, min(t.ctx, t.ctx - t.len + i + 1)) : t.ctx;
}
__device__ __forceinline__ int keys_from(const AttendParams& p, const Tile& t, int i) {
  return p.window ? min(t.ctx, max(0, max(0, t.ctx - t.len + i) - p.window + 1)) : 0;
}

// Tile j of a sequence whose number, first token, length and context are known.
__device__ __forceinline__ Tile finish_tile(const AttendParams& p, Tile t, int j, int group, int tile_rows) {
  t.rows = t.len * group;
  t.first = j * tile_rows;
  t.some = t.len > 0 && j >= 0 && t.first < t.rows;
  t.ctx = max(0, min(t.ctx, p.max_tokens));  // contexts end with the table
  if (!t.some) return t;
  const int t0 = t.first / group, t1 = min(t.len - 1, (t.first + tile_rows - 1) / group);
  t.hi = keys_to(p, t, t1);
  t.all_hi = keys_to(p, t, t0);
  t.all_lo = keys_from(p, t, t1);
  t.lo = keys_from(p, t, t0) & ~(kTok - 1);
  if (t.hi < t.lo) t.hi = t.lo;
  return t;
}

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
    const int lo = find_sequence(p.cu_seqlens, p.n_seqs, slot, [&](int64_t c, int n) { return c * group / tile_rows + n; });
    t.n = lo;
    j = slot - (int)((int64_t)cu[lo] * group / tile_rows + lo);
    t.begin = max(cu[lo], 0);
    t.len = (int)(min((int64_t)cu[lo + 1], p.tokens) - t.begin);
  }
  t.ctx = as_const(p.lens)[t.n];
  return finish_tile(p, t, j, group, tile_rows);
}

__device__ __forceinline__ int pieces(const AttendParams& p, const Tile& t) {
  return max(1, (t.hi - t.lo + p.piece - 1) / p.piece);
}

// A byte mask of the codes among four that are NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t m = ((w & 0x7f7f7f7fu) ^ 0x7f7f7f7fu) + 0x7f7f7f7fu;  // bit 7 of a byte set unless its code is NaN
  return (~m & 0x80808080u) >> 7;                                      // 1 where NaN
}

// A mask of the first n of 8 codes.
__device__ __forceinline__ uint2 first_codes(int n) {
  return make_uint2(n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1, n >= 8 ? 0xffffffffu : n <= 4 ? 0u : (1u << (8 * (n - 4))) - 1);
}
// NaN for the rows that see a NaN among 8 values of each lane: a product of ones
// (a code is NaN) and ones (the row sees tokens from .. to - 1).  0x38 is e4m3's 1.
template <typename T>
__device__ __forceinline__ void give_nan(uint2 nan, int from, int to, f32x4& o) {
  typedef Probs<T> P;
  float one[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) one[e] = e >= from && e < to ? 1.f : 0.f;
  typename P::vec see[P::N];
  P::make(one, see);
  const f32x4 hit = mfma(P::codes(nan.x * 0x38u, nan.y * 0x38u), see[0], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = hit[e] > 0.f ? __builtin_nanf("") : o[e];
}

// y * sigmoid(z)
template <typename T>
__device__ __forceinline__ float gated(float y, float z) { return y / (1.f + (sizeof(T) == 2 ? __expf(-z) : expf(-z))); }

// Four elements of an output row, gated where there is a gate.
template <typename T>
__device__ __forceinline__ void put(const AttendParams& p, f32x4 o, int64_t token, int64_t at) {
  float y[4] = {o[0], o[1], o[2], o[3]};
  if (p.gate) {
    float z[4];
    load4(reinterpret_cast<const T*>(p.gate) + token * p.gate_stride + at, z);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = gated<T>(y[e], z[e]);
  }
  store4(reinterpret_cast<T*>(p.o) + token * p.o_stride + at, y);
}

// The running maximum is that of score + log2 vscale, so that the weights, 2^(score - max) vscale, fit 16 bits; the
// sum of 2^(score - max) then ranges from 2^-120 to 2^98 with the scales.  The exponential gives no subnormals: it
// is taken 2^28 times as large, which brings terms of the smallest sum into its range and leaves the largest in it.
// A scale counts as 2^-90 at least: pages of zeros have the least there is.
constexpr float kUp = 28.f, kDown = 0x1p-28f;
__device__ __forceinline__ float log2_scale(float vs) { return fmaxf(__log2f(fabsf(vs)), -90.f); }
// From one maximum to a larger one: a sum l 2^x, where 2^x alone may be below fp32 (a page's sum is as large as its
// scale is small), and 2^x for the outputs.
__device__ __forceinline__ float lower(float& l, float x) {
  const float half = __builtin_amdgcn_exp2f(0.5f * x);
  l = l * half * half;
  return half * half;
}

// 16 bytes that nobody reads soon again: nontemporal (a decode step of 64 sequences of up to 32768 tokens 386 -> 364 us;
// fp32 queries, whose registers do not suffice, are the better without: 618 against 631).  Not so values of pages
// beyond 64 tokens, where two waves take the halves of a cache line (pages of 128, up to 16384 tokens: 297 -> 271 us).
template <bool STREAM>
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  if constexpr (!STREAM) return *reinterpret_cast<const uint4*>(p);
  const gdn_u4 w = __builtin_nontemporal_load(reinterpret_cast<const gdn_u4*>(p));
  return make_uint4(w.x, w.y, w.z, w.w);
}

// Shares: where every sequence has the same number of new tokens, all work is one line of steps of 256 tokens, tile
// after tile and head after head, and each of `shares` workgroups takes an equal length of it, whatever the
// contexts' lengths are.  Every workgroup finds the tiles' places on the line for itself (one pass over the
// lengths); the first leaves them for join_kernel.  A tile that several workgroups meet in has a partial result
// from each, at number (tile + workgroup), which rises along the line.
constexpr int kMostTiles = 2048;  // of a call that is cut into shares
constexpr int kStep = kWaves * kTok;
// (of fewer steps than workgroups each of the first gets one: every share in use has a step, so those that meet in a
// tile are numbered one after another)
__device__ __forceinline__ int64_t share_begin(const AttendParams& p, int64_t total, int64_t share) {
  const int64_t n = min((int64_t)p.shares, total);
  return min(share, n) * total / n;
}
__device__ __forceinline__ int share_of(const AttendParams& p, int64_t total, int64_t step) {
  return (int)(((step + 1) * min((int64_t)p.shares, total) - 1) / total);
}

// s_place[i]: steps of the tiles before tile i; their total after the last.  Called by all of a workgroup's waves.
__device__ __forceinline__ void place_tiles(const AttendParams& p, int group, int* s_place, int* s_sums) {
  const int per = (p.slots + kWaves * 64 - 1) / (kWaves * 64), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int slot = threadIdx.x * per + i;
    if (slot >= p.slots) break;
    Tile t;
    t.n = slot / p.uniform_tiles;
    t.len = (int)p.uniform;
    t.ctx = p.lens[t.n];
    t = finish_tile(p, t, slot - t.n * p.uniform_tiles, group, kRows);
    s_place[slot] = sum;
    sum += max(1, (t.hi - t.lo + kStep - 1) / kStep);
  }
  int before = sum;  // of this thread and those before it in its wave
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const int v = __shfl_up(before, x, 64);
    if (lane >= x) before += v;
  }
  if (lane == 63) s_sums[wave] = before;
  __syncthreads();
  before -= sum;
#pragma unroll
  for (int k = 0; k < kWaves; ++k)
    if (k < wave) before += s_sums[k];
  for (int i = 0; i < per; ++i) {
    const int slot = threadIdx.x * per + i;
    if (slot >= p.slots) break;
    s_place[slot] += before;
    if (slot == p.slots - 1) s_place[p.slots] = before + sum;
  }
  __syncthreads();
}

// WIDE: pages of more than 64 tokens.
template <typename T, int D, bool SHARES, bool WIDE>
__global__ __launch_bounds__(kWaves * 64, 2) void attend_kernel(AttendParams p) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int NQ = F32 ? 3 : 1;
  constexpr int KS = D / 32, MT = D / 16;
  typedef Probs<T> P;
  // the queries' operands through the loop, then the waves' outputs
  constexpr int kQBytes = KS * NQ * 64 * (int)sizeof(bf16x8), kOBytes = 2 * kRows * (D + 4) * (int)sizeof(float);
  __shared__ alignas(16) uint8_t lds[kQBytes > kOBytes ? kQBytes : kOBytes];
  __shared__ float s_m[kWaves][kRows], s_l[kWaves][kRows];
  bf16x8* s_q = reinterpret_cast<bf16x8*>(lds);
  float(*s_o)[kRows][D + 4] = reinterpret_cast<float(*)[kRows][D + 4]>(lds);

  __shared__ int s_place[SHARES ? kMostTiles + 1 : 1], s_sums[kWaves];
  const int group = p.h_q / p.h_kv;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int kg = r >> 2, ki = r & 3;  // this lane's row of the keys' operand: token 16 kg + 4 tt + ki
  const int in_page = (1 << p.page_shift) - 1;
  auto inside = [&](int id) { return id >= 0 && id < p.pages ? id : 0; };

  // what is left of this workgroup's share, in steps
  int64_t at = 0, end = 1, total = 1;
  if constexpr (SHARES) {
    place_tiles(p, group, s_place, s_sums);
    total = (int64_t)s_place[p.slots] * p.h_kv;
    at = share_begin(p, total, blockIdx.x), end = share_begin(p, total, (int64_t)blockIdx.x + 1);
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i <= p.slots; i += kWaves * 64) p.places[i] = s_place[i];
  }
  while (at < end) {
    int head = blockIdx.y, ns, start, stop;
    int64_t piece = blockIdx.z;  // which partial result this is
    Tile tile;
    if constexpr (SHARES) {
      int lo = 0, hi = p.slots - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)s_place[mid] * p.h_kv <= at) lo = mid; else hi = mid - 1;
      }
      const int slot = __builtin_amdgcn_readfirstlane(lo);
      const int steps = __builtin_amdgcn_readfirstlane(s_place[slot + 1] - s_place[slot]);
      const int64_t rest = at - (int64_t)__builtin_amdgcn_readfirstlane(s_place[slot]) * p.h_kv;
      head = (int)(rest / steps);
      const int step = (int)(rest - (int64_t)head * steps), n = (int)min((int64_t)(steps - step), end - at);
      tile = find_tile(p, slot, group, kRows);
      start = tile.lo + step * kStep;
      stop = min(tile.hi, start + n * kStep);
      ns = n == steps ? 1 : 2;  // the whole tile, or a part of it
      piece = (int64_t)slot * p.h_kv + head + blockIdx.x;
      at += n;
    } else {
      at = end;
      // workgroups go to the 8 XCDs in turn: every XCD gets pieces of every sequence, however unequal those are
      tile = find_tile(p, (blockIdx.x + blockIdx.z) % gridDim.x, group, kRows);
      if (!tile.some) return;
      ns = pieces(p, tile);
      if (piece >= ns) return;
      start = tile.lo + (int)piece * p.piece;
      stop = min(tile.hi, start + p.piece);
    }

    // A wave's codes stay on their way: a tile's keys are asked for when the last tile's have been used, and so
    // are its values; its pages a tile before that.
    const int32_t* table = p.page_table + (int64_t)tile.n * p.max_pages;
    // pages of this lane's 16 tokens as a row of the keys, and as a column of the scores
    auto page_of = [&](int token) { return token < stop ? table[token >> p.page_shift] : -1; };
    uint4 kc[4][D / 64], vc[MT];
    auto load_keys = [&](int k0, int pk) {
      const uint8_t* kp = p.k_cache + ((((int64_t)inside(pk) * p.h_kv + head) << p.page_shift) + ((k0 + 16 * kg) & in_page) + ki) * D + g * 16;
#pragma unroll
      for (int b = 0; b < D / 64; ++b)
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) kc[tt][b] = load_codes<!F32>(kp + tt * 4 * D + b * 64);
    };
    auto load_values = [&](int k0, int ps) {
      const uint8_t* vp = p.v_cache + ((((int64_t)inside(ps) * p.h_kv + head) * D + r) << p.page_shift) + ((k0 + 16 * g) & in_page);
#pragma unroll
      for (int i = 0; i < MT; ++i) vc[i] = load_codes<!F32 && !WIDE>(vp + ((i * 16) << p.page_shift));
    };
    const int k_first = start + wave * kTok;
    int pk = page_of(k_first + 16 * kg), ps = page_of(k_first + 16 * g);
    int pk_next = page_of(k_first + kStep + 16 * kg), ps_next = page_of(k_first + kStep + 16 * g);
    float ks = 0.f, vs = 0.f;
    if (k_first < stop) {
      load_keys(k_first, pk);
      load_values(k_first, ps);
      ks = p.k_scale[(int64_t)inside(ps) * p.h_kv + head], vs = p.v_scale[(int64_t)inside(ps) * p.h_kv + head];
    }

    // this lane's row
    const int row = tile.first + r;
    const bool live = row < tile.rows;  // the last tile's other rows see nothing and are not written
    const int tok = row / group, hq = head * group + (row - tok * group);
    const int row_hi = live ? keys_to(p, tile, tok) : 0, row_lo = keys_from(p, tile, tok);

    // Q: lane (row r, group g) holds elements 64 b + 16 g .. + 15 of each 64, the order its keys come in.  The
    // four waves make the operands together.
#pragma unroll
    for (int k = wave; k < KS; k += kWaves) {
      const int at = (k / 2) * 64 + g * 16 + (k & 1) * 8;
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) load8(reinterpret_cast<const T*>(p.q) + (tile.begin + tok) * p.q_stride + (int64_t)hq * D + at, f);
      bf16x8 q[NQ];
      if constexpr (F32) {
        split3_any(f, q);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[0][i] = (__bf16)f[i];
      }
#pragma unroll
      for (int i = 0; i < NQ; ++i) s_q[(k * NQ + i) * 64 + lane] = q[i];
    }
    __syncthreads();

    f32x4 o[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -__builtin_inff(), l = 0.f;

#pragma unroll 1
    for (int k0 = k_first; k0 < stop; k0 += kStep) {
      const int ts = k0 + 16 * g;
      const bool held = ps >= 0 && ps < p.pages;  // a page outside the pool holds nothing
      const bool more = k0 + kStep < stop;
      float ks_next = 0.f, vs_next = 0.f;
      if (more) ks_next = p.k_scale[(int64_t)inside(ps_next) * p.h_kv + head], vs_next = p.v_scale[(int64_t)inside(ps_next) * p.h_kv + head];

      f32x4 s[4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) s[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        bf16x8 q[2][NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) q[0][i] = s_q[(2 * b * NQ + i) * 64 + lane], q[1][i] = s_q[((2 * b + 1) * NQ + i) * 64 + lane];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const bf16x8 k_lo = to_bf16x8(kc[tt][b].x, kc[tt][b].y), k_hi = to_bf16x8(kc[tt][b].z, kc[tt][b].w);
#pragma unroll
          for (int i = NQ - 1; i >= 0; --i) {
            s[tt] = mfma(k_lo, q[0][i], s[tt]);
            s[tt] = mfma(k_hi, q[1][i], s[tt]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (more) load_keys(k0 + kStep, pk_next);
      __builtin_amdgcn_sched_barrier(0);

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
      float top = s[0][0];
#pragma unroll
      for (int e = 1; e < 15; e += 2) top = max3(top, s[e >> 2][e & 3], s[(e + 1) >> 2][(e + 1) & 3]);
      top = fmaxf(top, s[3][3]);
      // (the scales are positive, so the largest product is that of the largest score)
      top = sees ? fmaf(top, f, log2_scale(vs)) : -__builtin_inff();
      top = group_max(top);
      // the maximum moves only where it grows by more than 2^8: the weights then stay under 256
      if (__any(top > m + 8.f)) {
        const float now = fmaxf(m, top);
        const float alpha = lower(l, now == -__builtin_inff() ? now : m - now);
        m = now;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i] *= alpha;
      }
      const float base = (m == -__builtin_inff() ? 0.f : m) - kUp;
      float w[2][8];
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e >> 3][e & 7] = __builtin_amdgcn_exp2f(fmaf(s[e >> 2][e & 3], f, -base));
      if (part) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < from || e >= to) w[e >> 3][e & 7] = 0.f;
      }
      const float factor = sees ? vs * kDown : 0.f;  // whatever stands where no page is
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        l = fmaf(w[e >> 3][e & 7], kDown, l);
        w[e >> 3][e & 7] *= factor;
      }

      if (part) {
        // codes that must not reach the product: tokens behind the context or of no page, and NaN
        const int n = held ? tile.ctx - ts : 0;
        const uint2 keep[2] = {first_codes(n), first_codes(n - 8)};
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t* c = reinterpret_cast<uint32_t*>(&vc[i]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            c[2 * u] &= keep[u].x, c[2 * u + 1] &= keep[u].y;
            const uint2 bad = make_uint2(nan_bytes(c[2 * u]), nan_bytes(c[2 * u + 1]));
            if (__any((bad.x | bad.y) != 0)) {
              give_nan<T>(bad, from - 8 * u, to - 8 * u, o[i]);
              c[2 * u] &= ~(bad.x * 0xffu), c[2 * u + 1] &= ~(bad.y * 0xffu);
            }
          }
        }
      }
      typename P::vec pw[2][P::N];
      P::make(w[0], pw[0]);
      P::make(w[1], pw[1]);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const typename P::vec v_lo = P::codes(vc[i].x, vc[i].y), v_hi = P::codes(vc[i].z, vc[i].w);
#pragma unroll
        for (int e = P::N - 1; e >= 0; --e) {
          o[i] = mfma(v_lo, pw[0][e], o[i]);
          o[i] = mfma(v_hi, pw[1][e], o[i]);
        }
        if (i & 1) __builtin_amdgcn_sched_barrier(0);
      }
      if (more) load_values(k0 + kStep, ps_next);
      pk = pk_next, ps = ps_next, ks = ks_next, vs = vs_next;
      pk_next = page_of(k0 + 2 * kStep + 16 * kg), ps_next = page_of(k0 + 2 * kStep + 16 * g);
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);

    // Join the waves by their maxima and sums; rows pass through LDS two waves' at a time, so that two workgroups'
    // fit a CU with room to spare.
    __syncthreads();  // the queries have been read
    if (g == 0) s_m[wave][r] = m;
    __syncthreads();
    float mm = s_m[0][r];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) mm = fmaxf(mm, s_m[k][r]);
    const float a = lower(l, mm == -__builtin_inff() ? mm : m - mm);
    if (g == 0) s_l[wave][r] = l;
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i] *= a;
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
      if (live && (turn ? wave < 2 : wave >= 2)) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          f32x4* sum = reinterpret_cast<f32x4*>(&s_o[wave & 1][r][i * 16 + g * 4]);
          *sum = turn ? *sum + o[i] : o[i];
        }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < kRows * D / 4; i += kWaves * 64) {
      const int rr = i / (D / 4), c = (i - rr * (D / 4)) * 4, out_row = tile.first + rr;
      if (out_row >= tile.rows) break;
      float top = s_m[0][rr], ll = 0.f;
#pragma unroll
      for (int k = 1; k < kWaves; ++k) top = fmaxf(top, s_m[k][rr]);
#pragma unroll
      for (int k = 0; k < kWaves; ++k) ll += s_l[k][rr];
      const f32x4 sum = *reinterpret_cast<const f32x4*>(&s_o[0][rr][c]) + *reinterpret_cast<const f32x4*>(&s_o[1][rr][c]);
      const int64_t token = tile.begin + out_row / group;
      const int h = head * group + out_row % group;
      const int64_t out = token * p.h_q + h;
      if (ns == 1) {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        put<T>(p, sum * inv, token, (int64_t)h * D + c);
        if (p.lse && c == 0) p.lse[out] = ll == 0.f ? -__builtin_inff() : (top + __log2f(ll)) * 0.69314718055994530942f;
      } else {
        const int64_t part = SHARES ? piece * kRows + rr : piece * p.tokens * p.h_q + out;
        *reinterpret_cast<f32x4*>(p.part_o + part * D + c) = sum;
        if (c == 0) p.part_ml[2 * part] = top, p.part_ml[2 * part + 1] = ll;
      }
    }
    if constexpr (SHARES) __syncthreads();  // the next tile's queries take the sums' place
  }
}

// Long chunks: a workgroup's four waves take 32 rows each against the same
// keys and values.  A tile of 64 tokens, codes as they are, goes from memory
// to LDS without passing registers, one tile ahead of the products (two
// buffers, one barrier a tile); every wave turns the codes it reads into
// operands.  The products are 32x32x16 MFMAs: an MFMA of either size keeps
// vector instructions from issuing for about 8 of its cycles, and the larger
// one has twice as many to give.  Half a tile's scores S^T are 16 registers: a
// lane (row c, half h) holds those of 16 neighbouring tokens again, as keys
// are dealt to the operand's rows as token 16 (m >> 2 & 1) + 4 (m >> 3) + (m & 3).
// Sixteen-byte pieces are stored at places exclusive-ored with their row, so
// that the 16 rows that one read takes lie in different banks.
constexpr int kChunkRows = kWaves * 32;

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x16 zeros16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}
// The larger of lanes l and l ^ 32.
__device__ __forceinline__ float half_max(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// 16 bytes a lane from src + AT to dst + AT + 16 lane (dst: the wave's).
template <int AT>
__device__ __forceinline__ void to_lds(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)src,
                                   (__attribute__((address_space(3))) uint32_t*)dst, 16, AT, 0);
}
// The least and the largest of a wave's values, in a scalar register.
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = min(v, __shfl_xor(v, m, 64));
  return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ int wave_max(int v) { return -wave_min(-v); }

// What a tile of 64 tokens needs besides codes, for its four groups of 16 tokens (one where a page holds the
// whole tile): uniform, in scalar registers.
template <bool ONE>
struct TilePages {
  static constexpr int N = ONE ? 1 : 4;
  int id[N];
  float ks[N], vs[N];
  template <typename V>
  static __device__ __forceinline__ V of(const V (&v)[N], int g) {
    if constexpr (ONE) {
      return v[0];
    } else {
      const V lo = g & 1 ? v[1] : v[0], hi = g & 1 ? v[3] : v[2];
      return g & 2 ? hi : lo;
    }
  }
};

// ONE: a page holds at least 64 tokens.
template <typename T, int D, bool ONE>
__global__ __launch_bounds__(kWaves * 64, sizeof(T) == 4 && D == 256 ? 1 : 2) void attend_chunk_kernel(AttendParams p) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int NQ = F32 ? 3 : 1;
  constexpr int KB = D / 32, MT = D / 32, RS = D == 256 ? 0 : D == 128 ? 1 : 2;
  constexpr int kBytes = 2 * kTok * D;  // a tile: keys, then values
  typedef Probs<T> P;
  __shared__ alignas(16) uint8_t tiles[2 * kBytes];

  const int group = p.h_q / p.h_kv;
  // Workgroups go to the 8 XCDs in turn: a KV head's tiles go to as few as can share them evenly, whose L2
  // then holds that head's pages.  Later tiles see more keys: they begin first.
  const int turn_of = blockIdx.x >> 3, xcd = blockIdx.x & 7, piece = blockIdx.y;
  int head, slot;
  if (8 % p.h_kv == 0) {
    const int per = 8 / p.h_kv;
    head = xcd / per;
    slot = turn_of * per + xcd % per;
  } else {
    const int id = turn_of * 8 + xcd;
    head = id / p.slots;
    slot = id - head * p.slots;
  }
  if (slot >= p.slots || head >= p.h_kv) return;
  const Tile tile = find_tile(p, p.slots - 1 - slot, group, kChunkRows);
  if (!tile.some) return;
  const int ns = pieces(p, tile);
  if (piece >= ns) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 31, h = lane >> 5;

  int row_lo, row_hi;  // the keys that this lane's row sees
  bf16x8 q[2 * KB][NQ];
  {
    const int row = tile.first + wave * 32 + c;
    const bool live = row < tile.rows;
    const int tok = row / group, hq = head * group + (row - tok * group);
    row_hi = live ? keys_to(p, tile, tok) : 0;
    row_lo = live ? keys_from(p, tile, tok) : 0;
#pragma unroll
    for (int k = 0; k < 2 * KB; ++k) {
      const int at = (k / 2) * 32 + h * 16 + (k & 1) * 8;
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) load8(reinterpret_cast<const T*>(p.q) + (tile.begin + tok) * p.q_stride + (int64_t)hq * D + at, f);
      if constexpr (F32) {
        split3_any(f, q[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[k][0][i] = (__bf16)f[i];
      }
    }
  }
  f32x16 o[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) o[i] = zeros16();
  float m = -__builtin_inff(), l = 0.f;

  // what all of this wave's rows see (nothing, where one of them has no keys), and what any of them does
  const bool live_row = tile.first + wave * 32 + c < tile.rows;
  const int all_lo = wave_max(live_row ? row_lo : 0), all_hi = wave_min(live_row ? row_hi : INT32_MAX);
  const int any_lo = wave_min(live_row && row_hi > 0 ? row_lo : INT32_MAX), any_hi = wave_max(row_hi);

  const int start = tile.lo + piece * p.piece;
  const int stop = min(tile.hi, start + p.piece);
  const int in_page = (1 << p.page_shift) - 1;
  typedef TilePages<ONE> Pages;
  cint32* table = as_const(p.page_table + (int64_t)tile.n * p.max_pages);
  const __attribute__((address_space(4))) float* k_scale = (const __attribute__((address_space(4))) float*)(p.k_scale);
  const __attribute__((address_space(4))) float* v_scale = (const __attribute__((address_space(4))) float*)(p.v_scale);
  auto inside = [&](int id) { return id >= 0 && id < p.pages ? id : 0; };
  // (a group behind the last token takes the last token's page: its scores are masked)
  auto pages_of = [&](int k0, Pages& t) {
#pragma unroll
    for (int j = 0; j < Pages::N; ++j) t.id[j] = table[min(k0 + 16 * j, stop - 1) >> p.page_shift];
  };
  auto scales_of = [&](Pages& t) {
#pragma unroll
    for (int j = 0; j < Pages::N; ++j) {
      const int64_t at = (int64_t)inside(t.id[j]) * p.h_kv + head;
      t.ks[j] = k_scale[at];
      t.vs[j] = v_scale[at];
    }
  };
  // this lane's part of the tile's copy: keys of the 16 tokens of group `wave`, values of the tokens of group vg
  const int vg = (lane & 3) ^ (lane >> 4);
  const int krow = lane / (D / 16);
  const int k_from = krow * D + (((lane % (D / 16)) ^ (((krow & 7) | ((wave & 1) << 3)) >> RS)) * 16);
  const int v_from = ((lane >> 2) << p.page_shift) + (ONE ? 16 * vg : 0);
  auto stage = [&](int half, int k0, const Pages& t) {
    uint8_t* dst = tiles + half * kBytes + wave * (D * 16);
    const uint8_t* ks = p.k_cache + ((((int64_t)inside(Pages::of(t.id, wave)) * p.h_kv + head) << p.page_shift) + ((k0 + 16 * wave) & in_page)) * D;
    const uint8_t* vs = p.v_cache + ((((int64_t)inside(Pages::of(t.id, vg)) * p.h_kv + head) * D + wave * (D / 4)) << p.page_shift) +
                        ((k0 + (ONE ? 0 : 16 * vg)) & in_page);
    auto copy = [&](auto J) {
      constexpr int j = decltype(J)::value;
      // (1024 bytes on, a key of 256 is 4 rows on: its place's exclusive-or changes by 4 pieces every other time)
      to_lds<j * 1024>(ks + (D == 256 && (j & 1) ? k_from ^ 64 : k_from), dst);
      to_lds<0>(vs + v_from + ((16 * j) << p.page_shift), dst + kTok * D + j * 1024);
    };
    copy(std::integral_constant<int, 0>{});
    if constexpr (D > 64) copy(std::integral_constant<int, 1>{});
    if constexpr (D > 128) copy(std::integral_constant<int, 2>{}), copy(std::integral_constant<int, 3>{});
  };

  const int krow_c = 16 * ((c >> 2) & 1) + 4 * (c >> 3) + (c & 3);  // this lane's row of the keys' operand: its token
  const int key_at = krow_c * D + ((h ^ (((krow_c & 7) | ((krow_c >> 4) << 3)) >> RS)) * 16);
  const int value_at = kTok * D + c * 64 + ((h ^ ((c >> 2) & 3)) * 16);
  // A tile that some row of the workgroup does not see whole: codes that must not reach the products are cleared
  // in LDS, those of tokens behind the context or of no page, and NaN (which the rows that see one get here).
  auto clear = [&](int half, int k0, const Pages& pages) {
    uint8_t* values = tiles + half * kBytes + kTok * D;
    uint32_t bad = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < 4 * D; i += kWaves * 64) {
      const int of = (i & 3) ^ ((i >> 4) & 3), id = Pages::of(pages.id, of);
      const int n = id >= 0 && id < p.pages ? tile.ctx - k0 - 16 * of : 0;
      uint4* at = reinterpret_cast<uint4*>(values + i * 16);
      uint4 w = *at;
      const uint2 x = first_codes(n), y = first_codes(n - 8);
      w = make_uint4(w.x & x.x, w.y & x.y, w.z & y.x, w.w & y.y);
      bad |= nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w);
      *at = w;
    }
    if (!__syncthreads_or(bad != 0)) return;
    // a product of ones (a code is NaN; 0x38 is e4m3's 1) and ones (the row sees the token)
#pragma unroll 1
    for (int u = 0; u < 2; ++u) {
      const int lo = row_lo - (k0 + 32 * u + 16 * h), hi = row_hi - (k0 + 32 * u + 16 * h);
      float one[2][8];
#pragma unroll
      for (int e = 0; e < 16; ++e) one[e >> 3][e & 7] = e >= lo && e < hi ? 1.f : 0.f;
      typename P::vec see[2][P::N];
      P::make(one[0], see[0]);
      P::make(one[1], see[1]);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(tiles + half * kBytes + (value_at ^ (32 * u)) + i * 2048);
        const uint4 nan = make_uint4(nan_bytes(w.x) * 0x38u, nan_bytes(w.y) * 0x38u, nan_bytes(w.z) * 0x38u, nan_bytes(w.w) * 0x38u);
        f32x16 hit = mfma32(P::codes(nan.x, nan.y), see[0][0], zeros16());
        hit = mfma32(P::codes(nan.z, nan.w), see[1][0], hit);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = hit[e] > 0.f ? __builtin_nanf("") : o[i][e];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < 16 * D; i += kWaves * 64) {
      uint32_t* at = reinterpret_cast<uint32_t*>(values + i * 4);
      *at &= ~(nan_bytes(*at) * 0xffu);
    }
    __syncthreads();
  };

  // whole: every row of the wave sees every token of the tile
  auto compute = [&](bool whole, int half, int k0, const Pages& pages) {
    // Half a tile a turn (tokens 32 u .. + 31): its scores are half the registers
#pragma unroll 1
    for (int u = 0; u < 2; ++u) {
      const int ts = k0 + 32 * u + 16 * h;  // this lane's 16 tokens
      const int id = Pages::of(pages.id, 2 * u + h);
      const bool held = id >= 0 && id < p.pages;
      // (a scale of zero: scores of zero, and no 0 * infinity where they are masked)
      const float unit = Pages::of(pages.ks, 2 * u + h) * p.scale_log2, f = held ? (unit == 0.f ? 1e-30f : unit) : 1.f;
      const float vs = held ? Pages::of(pages.vs, 2 * u + h) : 1.f;

      f32x16 s = zeros16();
      const int keys = half * kBytes + 32 * u * D + key_at;
      auto key = [&](int b) { return *reinterpret_cast<const uint4*>(tiles + (keys ^ (b * 32))); };
      uint4 w4[2] = {key(0), key(1)};
#pragma unroll
      for (int b = 0; b < KB; b += 2) {
        uint4 next[2];
        if (b + 2 < KB) next[0] = key(b + 2), next[1] = key(b + 3);
        __builtin_amdgcn_sched_barrier(0);  // asked for before this step's products, not where registers come free
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w = w4[j >> 1];
          const bf16x8 kk = j & 1 ? to_bf16x8(w.z, w.w) : to_bf16x8(w.x, w.y);
#pragma unroll
          for (int i = NQ - 1; i >= 0; --i) s = mfma32(kk, q[2 * b + j][i], s);
        }
        if (b + 2 < KB) w4[0] = next[0], w4[1] = next[1];
        __builtin_amdgcn_sched_barrier(0);
      }
      if (!whole) {
        const int lo = row_lo - ts, hi = held ? row_hi - ts : 0;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < lo || e >= hi) s[e] = -__builtin_inff();
      }

      float top = fmaxf(s[0], s[1]);
#pragma unroll
      for (int e = 2; e < 16; e += 2) top = max3(top, s[e], s[e + 1]);
      top = half_max(fmaf(top, f, log2_scale(vs)));
      // the maximum moves only where it grows by more than 2^8: the weights then stay under 256
      if (__any(top > m + 8.f)) {
        const float now = fmaxf(m, top);
        const float alpha = lower(l, now == -__builtin_inff() ? now : m - now);
        m = now;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i] *= alpha;
      }
      const float base = (m == -__builtin_inff() ? 0.f : m) - kUp, factor = vs * kDown;
      typename P::vec pw[2][P::N];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] = __builtin_amdgcn_exp2f(fmaf(s[8 * j + e], f, -base));
          l = fmaf(w[e], kDown, l);
          w[e] *= factor;
        }
        P::make(w, pw[j]);
      }

      const int values = half * kBytes + (value_at ^ (32 * u));
      auto value = [&](int i) { return *reinterpret_cast<const uint4*>(tiles + values + i * 2048); };
      uint4 v[2] = {value(0), value(1)};
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < MT; i += 2) {
        uint4 next[2];
        if (i + 2 < MT) next[0] = value(i + 2), next[1] = value(i + 3);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const typename P::vec vv = j ? P::codes(v[x].z, v[x].w) : P::codes(v[x].x, v[x].y);
#pragma unroll
            for (int e = P::N - 1; e >= 0; --e) o[i + x] = mfma32(vv, pw[j][e], o[i + x]);
          }
        if (i + 2 < MT) v[0] = next[0], v[1] = next[1];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // A turn: the tile's codes have come (every wave waits for its own, then for the others'), the next tile's are
  // asked for, and the tile is worked through.
  Pages here, next;
  if (start < stop) {
    pages_of(start, here);
    stage(0, start, here);
    scales_of(here);
    pages_of(start + kTok, next);
  }
  int half = 0;
#pragma unroll 1
  for (int k0 = start; k0 < stop; k0 += kTok) {
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __syncthreads();
    if (k0 + kTok < stop) {
      stage(half ^ 1, k0 + kTok, next);
      scales_of(next);
    }
    bool there = true;
#pragma unroll
    for (int j = 0; j < Pages::N; ++j) there = there && here.id[j] >= 0 && here.id[j] < p.pages;
    if (!(there && k0 >= tile.all_lo && k0 + kTok <= tile.all_hi)) clear(half, k0, here);
    if (k0 < any_hi && k0 + kTok > any_lo) compute(there && k0 >= all_lo && k0 + kTok <= all_hi, half, k0, here);
    here = next;
    pages_of(k0 + 2 * kTok, next);
    half ^= 1;
  }

  int row = tile.first + wave * 32 + c;
  asm volatile("" : "+v"(row));  // what follows is worked out here, not kept through the loop
  l += __shfl_xor(l, 32, 64);
  if (row >= tile.rows) return;
  const int64_t token = tile.begin + row / group;
  const int hq = head * group + row % group;
  const int64_t out = token * p.h_q + hq;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int at = i * 32 + 8 * a + 4 * h;
      const f32x4 y = f32x4{o[i][4 * a], o[i][4 * a + 1], o[i][4 * a + 2], o[i][4 * a + 3]};
      if (ns == 1) put<T>(p, y * inv, token, (int64_t)hq * D + at);
      else *reinterpret_cast<f32x4*>(p.part_o + ((int64_t)piece * p.tokens * p.h_q + out) * D + at) = y;
    }
  if (h) return;
  if (ns > 1) {
    const int64_t part = (int64_t)piece * p.tokens * p.h_q + out;
    p.part_ml[2 * part] = m, p.part_ml[2 * part + 1] = l;
  } else if (p.lse) {
    p.lse[out] = l == 0.f ? -__builtin_inff() : (m + __log2f(l)) * 0.69314718055994530942f;
  }
}

// Joins the pieces of a row, its lanes over the head's elements, eight pieces at a time on their way.  Where there may
// be more than eight a workgroup's four waves share a row (one token over 32768 in 128 pieces: 24 us in all, 45 with one
// piece after another), otherwise each has its own (538 tokens of 32 heads of 256 in up to 4
// pieces: 18 us, 47 with a workgroup a row).
constexpr int kJoin = 8;
template <typename T, int D, bool SHARES>
__global__ __launch_bounds__(kWaves * 64) void join_kernel(AttendParams p) {
  constexpr int E = D / 64;
  __shared__ float s_sum[kWaves][D], s_l[kWaves];
  const int group = p.h_q / p.h_kv, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Tile tile = find_tile(p, blockIdx.x, group, p.tile_rows);
  if (!tile.some) return;
  const int share = p.join_waves == 1 ? 0 : wave, at = tile.first + (p.join_waves == 1 ? (int)blockIdx.z * kWaves + wave : (int)blockIdx.z);
  int ns;
  int64_t part0 = 0;  // the first partial result's row
  if constexpr (SHARES) {
    const int64_t total = (int64_t)p.places[p.slots] * p.h_kv;
    const int from = p.places[blockIdx.x], steps = p.places[blockIdx.x + 1] - from;
    const int64_t begin = (int64_t)from * p.h_kv + (int64_t)blockIdx.y * steps;
    const int first = share_of(p, total, begin);
    ns = share_of(p, total, begin + steps - 1) - first + 1;
    part0 = ((int64_t)blockIdx.x * p.h_kv + blockIdx.y + first) * kRows + (at - tile.first);
  } else {
    ns = pieces(p, tile);
  }
  if (ns == 1 || at >= tile.rows) return;  // written already, or no row
  const int64_t token = tile.begin + at / group;
  const int h = blockIdx.y * group + at % group;
  const int64_t out = token * p.h_q + h, step = SHARES ? kRows : p.tokens * p.h_q;
  if (!SHARES) part0 = out;
  float mm = -__builtin_inff();
  for (int s = lane; s < ns; s += 64) mm = fmaxf(mm, p.part_ml[2 * (s * step + part0)]);
#pragma unroll
  for (int x = 32; x >= 1; x >>= 1) mm = fmaxf(mm, __shfl_xor(mm, x, 64));
  const float base = mm == -__builtin_inff() ? 0.f : mm;
  float sum[E], ll = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.f;
  for (int s0 = share; s0 < ns; s0 += p.join_waves * kJoin) {
    float row[kJoin][E], ml[kJoin][2];
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      const int64_t part = min(s0 + j * p.join_waves, ns - 1) * step + part0;
      ml[j][0] = p.part_ml[2 * part], ml[j][1] = p.part_ml[2 * part + 1];
#pragma unroll
      for (int e = 0; e < E; ++e) row[j][e] = p.part_o[part * D + lane * E + e];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      const bool there = s0 + j * p.join_waves < ns;  // (those behind the last are the last again)
      const float f = lower(ml[j][1], ml[j][0] - base), a = there ? f : 0.f;
      ll += there ? ml[j][1] : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] = fmaf(a, row[j][e], sum[e]);
    }
  }
  if (p.join_waves == 1) {
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int64_t c = (int64_t)h * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float y = sum[e] * inv;
      if (p.gate) y = gated<T>(y, to_f32(reinterpret_cast<const T*>(p.gate)[token * p.gate_stride + c + e]));
      reinterpret_cast<T*>(p.o)[token * p.o_stride + c + e] = from_f32<T>(y);
    }
    if (p.lse && lane == 0) p.lse[out] = ll == 0.f ? -__builtin_inff() : (mm + __log2f(ll)) * 0.69314718055994530942f;
    return;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_sum[wave][lane * E + e] = sum[e];
  if (lane == 0) s_l[wave] = ll;
  __syncthreads();
  ll = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  if (threadIdx.x < D) {
    const int64_t c = (int64_t)h * D + threadIdx.x;
    float y = ((s_sum[0][threadIdx.x] + s_sum[1][threadIdx.x]) + (s_sum[2][threadIdx.x] + s_sum[3][threadIdx.x])) * inv;
    if (p.gate) y = gated<T>(y, to_f32(reinterpret_cast<const T*>(p.gate)[token * p.gate_stride + c]));
    reinterpret_cast<T*>(p.o)[token * p.o_stride + c] = from_f32<T>(y);
  }
  if (p.lse && threadIdx.x == 0) p.lse[out] = ll == 0.f ? -__builtin_inff() : (mm + __log2f(ll)) * 0.69314718055994530942f;
}

// How a call is cut: tiles of rows, and pieces of the context of `piece` tokens.
struct Plan {
  bool chunk;      // attend_chunk_kernel
  int32_t tile_rows;
  int64_t slots;  // tiles at most
  int32_t uniform_tiles;
  int64_t uniform;
  int32_t piece;
  int64_t pieces;  // of the longest context that the table holds
  int32_t shares;  // 0: pieces
  int32_t join_waves;  // that join a row
  int64_t parts;   // rows of partial results
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
  // Rows of 128 share their keys among a workgroup's waves where a sequence has at least two tiles of 16 (averages;
  // 32 sequences of 4096 tokens, 4 heads of 256: 73 against 85 us with 12 rows, 110 against 89 with 24), and all of
  // them enough for that kernel's fewer and longer workgroups (one sequence of 8192: 38 against 36 us with 24 tiles in
  // all, 24 against 35 with 8).  In fp32 the chunk kernel holds the queries as three times as many registers, half the
  // waves: from three tiles with heads of 256 (150 against 205 us, 257 against 216 with 36 rows), from 400 rows with
  // smaller ones (one sequence of 8192, heads of 128: 42 against 44 us with 288 rows, 110 against 100 with 1200).
  const double rows = (double)a.tokens * group / a.n_seqs, all = a.n_seqs * std::ceil(rows / kRows) * a.h_kv;
  const int least = a.bf16 ? kRows : a.d == 256 ? 2 * kRows : 400;
  c.chunk = rows > least && all >= (a.d == 256 ? 24 : 32);
  c.tile_rows = !c.chunk ? kRows : kChunkRows;
  c.uniform_tiles = (int32_t)((c.uniform * group + c.tile_rows - 1) / c.tile_rows);
  c.slots = a.ragged ? a.tokens * group / c.tile_rows + a.n_seqs : (int64_t)c.uniform_tiles * a.n_seqs;
  // Pieces of the contexts, for enough workgroups: of single tokens about 4096 (16 for each CU), of chunks at most 512, as
  // many as run at once (one sequence of 8192, 4 heads of 256: 1200 rows take 81 us, 94 in 1024 pieces; two of 4000 with
  // 7800 rows, 488 tiles, 251 us whole, 382 in twice as many).  Both of at least 256 tokens, a turn of the waves of a workgroup with single tokens (102 rows: 32 us,
  // 39 with 512).
  // (a causal window bounds the keys of a tile: those of its first token's window to its last token)
  int64_t most = max_tokens(a);
  if (a.causal && a.window > 0) most = std::min(most, (int64_t)a.window + (c.tile_rows - 1) / group + kTok);
  const int64_t step = kStep, tiles = c.slots * a.h_kv;
  int64_t piece = (int64_t)std::min((double)most, (double)most * tiles / 4096);
  // Short contexts whole, which saves the second launch: up to 1024 tokens (one token, 8 heads of 128: 9.0 us, 11.8 in
  // pieces; of 64 sequences, 8 heads of 64: 14.4 and 20.7), with heads of 256 up to 512 unless there is a tile for
  // every CU (one token of 16 sequences, 4 heads: 15.9 and 16.4 us over 512, 24.5 and 16.4 over 1024; of 64: 27.8 and
  // 36).
  const int64_t whole = a.d == 256 && tiles < 256 ? 512 : 1024;
  if (most <= whole) piece = most;
  if (c.chunk) piece = tiles < 512 ? (most + 512 / tiles - 1) / (512 / tiles) : most;
  piece = (piece + step - 1) / step * step;
  c.piece = (int32_t)(piece < step ? step : piece);
  c.pieces = (most + c.piece - 1) / c.piece;
  if (c.pieces < 1) c.pieces = 1;
  // Shares instead, as many as run at once (2 workgroups to each of 256 CUs; 4 with heads of 64, 3 in fp32), where
  // the longest contexts would give each at least 4 steps.
  const int64_t at_once = 256 * (a.d != 64 ? 2 : a.bf16 ? 4 : 3);
  c.shares = 0;
  const int64_t steps = c.slots * ((most + kStep - 1) / kStep);  // of one head, added up in 32 bits
  if (!c.chunk && !a.ragged && c.slots <= kMostTiles && steps <= INT32_MAX && steps * a.h_kv >= 4 * at_once) c.shares = (int32_t)at_once;
  c.join_waves = (c.shares ? c.shares / tiles : c.pieces) > 8 ? kWaves : 1;
  c.parts = c.shares ? (c.shares + tiles) * kRows : c.pieces > 1 ? c.pieces * a.tokens * a.h_q : 0;
  return c;
}

template <typename T, int D>
hipError_t launch(const AttendParams& p, const Plan& c, hipStream_t stream) {
  const int64_t rows = p.cu_seqlens ? c.tile_rows : std::min((int64_t)c.tile_rows, c.uniform * (p.h_q / p.h_kv));
  const dim3 block(kWaves * 64), joins((unsigned)c.slots, (unsigned)p.h_kv, (unsigned)(p.join_waves == 1 ? (rows + kWaves - 1) / kWaves : rows));
  constexpr bool kWide = sizeof(T) == 2;  // fp32 has one form
  const bool wide = kWide && p.page_shift > 6;
  if (c.shares) {
    if (wide) hipLaunchKernelGGL((attend_kernel<T, D, true, kWide>), dim3((unsigned)c.shares), block, 0, stream, p);
    else hipLaunchKernelGGL((attend_kernel<T, D, true, false>), dim3((unsigned)c.shares), block, 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((join_kernel<T, D, true>), joins, block, 0, stream, p);
    return hipGetLastError();
  }
  const int64_t turns = (c.slots * p.h_kv + 7) / 8;
  if (turns > INT32_MAX / 8) return hipErrorInvalidValue;
  const dim3 grid((unsigned)c.slots, (unsigned)p.h_kv, (unsigned)c.pieces), chunks((unsigned)(turns * 8), (unsigned)c.pieces);
  if (!c.chunk && wide) hipLaunchKernelGGL((attend_kernel<T, D, false, kWide>), grid, block, 0, stream, p);
  else if (!c.chunk) hipLaunchKernelGGL((attend_kernel<T, D, false, false>), grid, block, 0, stream, p);
  else if (p.page_shift >= 6) hipLaunchKernelGGL((attend_chunk_kernel<T, D, true>), chunks, block, 0, stream, p);
  else hipLaunchKernelGGL((attend_chunk_kernel<T, D, false>), chunks, block, 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || c.pieces == 1) return e;
  hipLaunchKernelGGL((join_kernel<T, D, false>), joins, block, 0, stream, p);
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
  if (!c.parts) return 0;
  return round256(c.parts * a.d * sizeof(float)) + round256(c.parts * 2 * sizeof(float)) + (c.shares ? round256((c.slots + 1) * sizeof(int)) : 0);
}

hipError_t launch_attend(AttendParams p, const AttendShape& a, void* workspace, int dtype, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  const Plan c = plan(a);
  p.max_tokens = max_tokens(a);
  p.uniform = c.uniform;
  p.uniform_tiles = c.uniform_tiles;
  p.piece = c.piece;
  p.tile_rows = c.tile_rows;
  p.slots = (int32_t)c.slots;
  p.shares = c.shares;
  p.join_waves = c.join_waves;
  if (c.parts) {
    char* w = reinterpret_cast<char*>(workspace);
    p.part_o = reinterpret_cast<float*>(w);
    w += round256(c.parts * a.d * sizeof(float));
    p.part_ml = reinterpret_cast<float*>(w);
    p.places = reinterpret_cast<int32_t*>(w + round256(c.parts * 2 * sizeof(float)));
  }
  return dtype == 1 ? launch_d<__bf16>(p, c, a.d, stream) : launch_d<float>(p, c, a.d, stream);
}

}  // namespace gdn
