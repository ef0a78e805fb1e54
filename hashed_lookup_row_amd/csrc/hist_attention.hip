// Attention over the 8-bit history cache: out = softmax(s q K^T) V for ragged
// requests, with keys and values as codes times a scale per block and head.
//
// Everything one wave does is a tile of 64 tokens (four chunks of 16) against
// 16 query rows, in registers:
//   S^T = K Q^T   v_mfma_f32_16x16x32_f16, A = codes as f16 (exact: they are
//                 whole numbers up to 127), B = the queries
//   O^T = V^T P^T with the scores' own registers as the B operand
// The tokens that lane group g (= lane/16) holds after the first product are
// exactly chunk g: the rows of the A operand are given to lanes in the order
// token(t, m) = 16 (m/4) + 4 t + m%4, so the second product's operand needs no
// exchange between lanes, and each lane has one key scale and one value scale
// (a block holds whole chunks).  A lane's value operand for one d is the 16
// bytes of [chunk][d][16].
//
// Precision: a query row is multiplied by a power of two that brings its
// largest magnitude to [512, 1024), so elements of bf16 and f16 queries down to
// 2^-23 of it are exact in f16, smaller ones off by at most 2^-34 of it (fp32 ones
// are split into two f16 parts, 22 bits).  Scores, the running maximum and
// sum, and the output are fp32.  The weights p are one f16 part for bf16
// outputs (the error against 64 bits is 1.671e-3 with one and 1.660e-3, the output's own
// rounding, with two, which take 29% longer in a causal prompt and 41% for candidates) and two for
// fp16 and fp32: at 11 bits their own rounding would be as
// large as fp16's (the error against 64 bits 1.4 to 1.5 times what the output's rounding gives).  A
// weight enters the second product times its chunk's value scale, relative to
// the row's largest such product so far and times 2^12, which keeps terms
// down to 2^-23 of the largest in f16's normal range.  Running maxima are whole
// numbers (in log2), so rescaling and joining waves and splits is exact.
#include "hlr_common.hpp"
#include "hist_common.hpp"

#include <type_traits>

namespace {
using namespace hlr;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 64;      // tokens of a tile
constexpr int kWaves = 4;      // waves of a block
constexpr float kNone = -3.0e38f;  // running maxima of a row that has seen nothing
constexpr float kUp = 12.f;    // weights are held as 2^kUp p
constexpr float kSlack = 3.f;  // a running maximum follows once scores pass it by this (in log2)

struct Args {
  const void *q;
  int64_t q_tok, q_head;  // strides, elements
  const int8_t *k, *v;
  const float *ks, *vs;
  const int *table;
  int64_t cols;
  const int *lengths, *cu;
  void *out;
  float *lse;        // nullable
  float *part;       // [splits][tokens][heads][D], when split
  float2 *part_ml;   // [splits][tokens][heads]: running maximum and sum
  int64_t tokens, num_blocks;
  int kv_heads, group, log_b;
  int causal, window;
  float scale;       // softmax scale times log2(e)
  int chunk;         // tokens of a split
  int row_tiles;     // blocks of rows per request
  uint32_t requests, splits;
  int max_q, max_len;  // the caller's bounds: what a launch covers
};

// The first position that a query at position `at` (below 0: before the history's first) sees through the window;
// no difference is taken that passes 32 bits, whatever the window.
__device__ __forceinline__ int first_seen(const Args &a, int at) { return at >= a.window ? at + 1 - a.window : 0; }

__device__ __forceinline__ h8 f16_of_codes(uint32_t lo, uint32_t hi) {
  // byte b -> f16 with bits 0x64xx = 1024 + (b ^ 0x80) = 1152 + code
  lo ^= 0x80808080u;
  hi ^= 0x80808080u;
  const uint32_t w[4] = {
      __builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u), __builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u),
      __builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u), __builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u)};
  const h2 bias = {static_cast<_Float16>(1152.f), static_cast<_Float16>(1152.f)};
  h8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const h2 x = __builtin_bit_cast(h2, w[i]) - bias;
    r[2 * i] = x[0];
    r[2 * i + 1] = x[1];
  }
  return r;
}

__device__ __forceinline__ float xor16(float x) { return __shfl_xor(x, 16); }
__device__ __forceinline__ float xor32(float x) { return __shfl_xor(x, 32); }

// 2^d for a whole number d, held within what fp32 can scale by.
__device__ __forceinline__ float pow2(float d) {
  return ldexpf(1.f, static_cast<int>(fminf(fmaxf(d, -200.f), 126.f)));
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -__builtin_inff() : __builtin_fmaf(m, 0.693147180559945309f, logf(ldexpf(l, -static_cast<int>(kUp))));
}

// A tile of 64 tokens as f16 in LDS, in units of 16 bytes: keys as rows (t, m)
// of D/8 units, token(t, m) as above; values as rows d of 8 units (unit 2 g + u:
// tokens 8 u .. 8 u + 7 of chunk g).  A read takes one unit of 16
// successive rows; the units of a row are permuted (xor) so that those of eight
// successive rows lie in different banks.  (Conflicts still take 24 to 38% of the LDS's
// cycles, so a 16-byte access does not go by eight neighbouring lanes alone.)
template <int D>
struct RowTile {  // D = 64, 128, 256
  static constexpr int kUnits = D / 8, kKeys = 64 * kUnits, kValues = D * 8;  // units of a key row, of both tiles
  static __device__ __forceinline__ int key_at(int t, int m, int unit) {
    return (t * 16 + m) * kUnits + (unit ^ (m & (kUnits - 1)));
  }
  static __device__ __forceinline__ int value_at(int d, int unit) { return d * 8 + (unit ^ (d & 7)); }
};

// One wave's state for NQ tiles of 16 rows.
template <typename T, int D, int NQ>
struct Wave {
  static constexpr int NP = sizeof(T) == 4 ? 2 : 1;                  // f16 parts of a query
  static constexpr int NW = std::is_same<T, bf16>::value ? 1 : 2;  // f16 parts of a weight
  static constexpr int NC = D / 32;               // products of 32 elements
  static constexpr int ND = D / 16;               // output tiles of 16 elements
  static constexpr int NK = D >= 64 ? D / 64 : 1; // 16-byte loads of a key row per lane (8 bytes for D = 32)
  h8 q[NQ][NP][NC];
  f4 acc[NQ][ND];
  float m[NQ], m2[NQ], rel[NQ], l[NQ], qs[NQ];
  int hi[NQ], lo[NQ];  // the row sees positions lo <= p < hi

  __device__ __forceinline__ void load_queries(const Args &a, int r, int kvh, int row0, int rows, int first_token,
                                               int fresh, int length) {
    const int lane = lane_id(), n = lane % 16, g = lane / 16;
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
      const int row = row0 + 16 * x + n;
      const bool real = row < rows;
      const int i = real ? row / a.group : 0, head = kvh * a.group + (real ? row % a.group : 0);
      const T *p = static_cast<const T *>(a.q) + (first_token + i) * a.q_tok + head * a.q_head;
      float v[NC][8];
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d = D >= 64 ? (c / 2) * 64 + g * 16 + (c % 2) * 8 : g * 8;
        // rows past the end read a real row's elements and drop them
        T y[8];
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<u4 *>(y) = *reinterpret_cast<const u4 *>(p + d);
          *reinterpret_cast<u4 *>(y + 4) = *reinterpret_cast<const u4 *>(p + d + 4);
        } else {
          *reinterpret_cast<u4 *>(y) = *reinterpret_cast<const u4 *>(p + d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[c][j] = real ? static_cast<float>(y[j]) : 0.f;
          top = fmaxf(top, fabsf(v[c][j]));
        }
      }
      top = fmaxf(top, xor16(top));
      top = fmaxf(top, xor32(top));
      int e = 0;
      if (top > 0.f && top <= 3.402823466e38f) e = 9 - ilogbf(top);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = a.scale < 0.f ? -ldexpf(v[c][j], e) : ldexpf(v[c][j], e);  // scales in weights() are not negative
          q[x][0][c][j] = static_cast<_Float16>(y);
          if constexpr (NP == 2) q[x][1][c][j] = static_cast<_Float16>(y - static_cast<float>(q[x][0][c][j]));
        }
      qs[x] = ldexpf(fabsf(a.scale), -e);
      hi[x] = 0;
      lo[x] = 0;
      if (real) {
        hi[x] = length;
        if (a.causal) {
          const int at = length - fresh + i;
          hi[x] = max(at + 1, 0);
          if (a.window > 0) lo[x] = first_seen(a, at);
        }
      }
      m[x] = m2[x] = kNone;
      rel[x] = 1.f;
      l[x] = 0.f;
#pragma unroll
      for (int e2 = 0; e2 < ND; ++e2) acc[x][e2] = f4{0.f, 0.f, 0.f, 0.f};
    }
  }

  // One tile: kr, vr the raw codes, ks/vs the scales of this lane's chunk
  // (chunk ok: the lane's own chunk has a block), base the tile's position.
  __device__ __forceinline__ void scores(const u4 (&kr)[4][NK], f4 (&s)[NQ][4]) const {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int x = 0; x < NQ; ++x) s[x][t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const u4 w = kr[t][c / 2];
        const h8 kf = (c % 2) ? f16_of_codes(w[2], w[3]) : f16_of_codes(w[0], w[1]);
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
          for (int p = 0; p < NP; ++p) s[x][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[x][p][c], s[x][t], 0, 0, 0);
      }
    }
  }

  // The products from f16 tiles in LDS (RowTile below), K's rows in the order
  // of the A operand.
  __device__ __forceinline__ void scores(const u4 *kt, f4 (&s)[NQ][4]) const {
    const int lane = lane_id(), n = lane % 16, g = lane / 16;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int x = 0; x < NQ; ++x) s[x][t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int unit = (c / 2) * 8 + 2 * g + c % 2;
        const h8 kf = __builtin_bit_cast(h8, kt[RowTile<D>::key_at(t, n, unit)]);
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
          for (int p = 0; p < NP; ++p) s[x][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[x][p][c], s[x][t], 0, 0, 0);
      }
    }
  }

  __device__ __forceinline__ void values(const u4 *vt, const f4 (&s)[NQ][4]) {
    const int lane = lane_id(), n = lane % 16, g = lane / 16;
    h8 p[NQ][NW][2];
    weights16(s, p);
#pragma unroll
    for (int e = 0; e < ND; ++e)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const h8 vf = __builtin_bit_cast(h8, vt[RowTile<D>::value_at(e * 16 + n, 2 * g + u)]);
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
          for (int k = 0; k < NW; ++k) acc[x][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[x][k][u], acc[x][e], 0, 0, 0);
      }
  }

  // Masks the scores, keeps the running maxima (m of the scores, m2 of the scores times the value scales, both in
  // log2 and whole numbers, so every rescaling is exact), adds up l and leaves the weights times the value scales in
  // s.  Maxima are compared per lane and joined over the lane groups only when some lane passes them by kSlack; a row
  // follows its own scores alone.
  __device__ __forceinline__ void weights(f4 (&s)[NQ][4], float ks, float vs, bool ok, int base) {
    const int g = lane_id() / 16;
    if (!ok) ks = 0.f, vs = 0.f;
    const float ev = vs > 0.f ? static_cast<float>(__builtin_amdgcn_frexp_expf(vs)) : -__builtin_inff();
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
      float f = ks * qs[x];
      const bool whole = base >= lo[x] && base + kTile <= hi[x] && ok;
      if (ballot(!whole)) {
        const int p0 = base + 16 * g;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int p = p0 + 4 * t + i;
            s[x][t][i] = (ok && p >= lo[x] && p < hi[x]) ? s[x][t][i] * f : -__builtin_inff();
          }
        f = 1.f;
      }
      float top = s[x][0][0];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[x][t][i]);
      top *= f;
      if (ballot(top > m[x] + kSlack || top + ev > m2[x] + kSlack)) {
        float top2 = top + ev;
        top = fmaxf(top, xor16(top));
        top = fmaxf(top, xor32(top));
        top2 = fmaxf(top2, xor16(top2));
        top2 = fmaxf(top2, xor32(top2));
        const float now = top > m[x] + kSlack ? __builtin_ceilf(top) : m[x];
        const float now2 = top2 > m2[x] + kSlack ? __builtin_ceilf(top2) : m2[x];
        l[x] *= pow2(m[x] - now);
        const float by = pow2(m2[x] - now2);
#pragma unroll
        for (int e = 0; e < ND; ++e) acc[x][e] *= by;
        m[x] = now;
        m2[x] = now2;
        rel[x] = pow2(now - now2);
      }
      // finite where p is 0: the best scores' values may all be zero (a scale of 0, m far above m2), and the scale of a
      // block that the row sees nothing of may be anything
      const float off = kUp - m[x], c = __builtin_amdgcn_fmed3f(vs * rel[x], -3.402823466e38f, 3.402823466e38f);
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][t][i], f, off));
          sum += p;
          s[x][t][i] = p * c;
        }
      l[x] += sum;
    }
  }

  // The B operand of the second product: the weights as f16, in one part or two.
  __device__ __forceinline__ void weights16(const f4 (&s)[NQ][4], h8 (&p)[NQ][NW][2]) const {
#pragma unroll
    for (int x = 0; x < NQ; ++x)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float y = s[x][2 * u + j / 4][j % 4];
          // the product's fp32 rounding has to happen before both parts are taken: without this the first
          // part is rounded to f16 straight from the product, and at ties the two parts disagree
          if constexpr (NW == 2) asm("" : "+v"(y));
          p[x][0][u][j] = static_cast<_Float16>(y);
          if constexpr (NW == 2) p[x][1][u][j] = static_cast<_Float16>(y - static_cast<float>(p[x][0][u][j]));
        }
  }

  __device__ __forceinline__ void values(const u4 (&vr)[ND], const f4 (&s)[NQ][4]) {
    h8 p[NQ][NW][2];
    weights16(s, p);
#pragma unroll
    for (int e = 0; e < ND; ++e)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const h8 vf = u ? f16_of_codes(vr[e][2], vr[e][3]) : f16_of_codes(vr[e][0], vr[e][1]);
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
          for (int k = 0; k < NW; ++k) acc[x][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[x][k][u], acc[x][e], 0, 0, 0);
      }
  }
};

// The block ids of a lane: `own` for its chunk lane/16 (scales, values), `row`
// for the key rows it loads (chunk (lane%16)/4).
struct Ids {
  int own, row;
};

__device__ __forceinline__ int block_of(const Args &a, const int *table, int pos) {
  const int64_t col = pos >> a.log_b;
  int b = -1;
  if (col < a.cols) b = table[col];
  return b >= 0 && b < a.num_blocks ? b : -1;
}

__device__ __forceinline__ Ids ids_of(const Args &a, const int *table, int tile) {
  const int lane = lane_id(), base = tile * kTile;
  return Ids{block_of(a, table, base + 16 * (lane / 16)), block_of(a, table, base + 16 * (lane % 16 / 4))};
}

// The raw codes of a tile's keys: row token(t, m) of the A operand, 16 bytes
// of 64 (or 8 of 32) elements per lane.  Lanes without a block read block 0.
template <int D, int NK>
__device__ __forceinline__ void load_keys(const Args &a, Ids id, int kvh, int tile, u4 (&kr)[4][NK]) {
  const int lane = lane_id(), n = lane % 16, g = lane / 16;
  const int at = (tile * kTile + 16 * (n / 4) + n % 4) & ((1 << a.log_b) - 1);
  const int8_t *p =
      a.k + (((static_cast<int64_t>(max(id.row, 0)) * a.kv_heads + kvh) << a.log_b) + at) * D + g * (D >= 64 ? 16 : 8);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if constexpr (D >= 64) {
#pragma unroll
      for (int c = 0; c < NK; ++c) kr[t][c] = *reinterpret_cast<const u4 *>(p + t * 4 * D + c * 64);
    } else {
      const u2 y = *reinterpret_cast<const u2 *>(p + t * 4 * D);
      kr[t][0] = u4{y[0], y[1], 0u, 0u};
    }
  }
}

// The raw codes of a tile's values (16 tokens of one element per load) and
// the scales of this lane's chunk.
template <int D, int ND>
__device__ __forceinline__ void load_values(const Args &a, Ids id, int kvh, int tile, u4 (&vr)[ND], float &ks, float &vs) {
  const int lane = lane_id(), n = lane % 16, g = lane / 16;
  const int chunk = ((tile * kTile + 16 * g) & ((1 << a.log_b) - 1)) >> 4;
  const int64_t bh = static_cast<int64_t>(max(id.own, 0)) * a.kv_heads + kvh;
  const int8_t *p = a.v + (((bh << (a.log_b - 4)) + chunk) * D + n) * 16;
#pragma unroll
  for (int e = 0; e < ND; ++e) vr[e] = *reinterpret_cast<const u4 *>(p + e * 256);
  ks = a.ks[bh];
  vs = a.vs[bh];
}

// A request's length, within what the launch covers: where its queries stand.
__device__ __forceinline__ int length_of(const Args &a, int r) { return max(0, min(a.lengths[r], a.max_len)); }

// Its positions that the table row has a place for; later ones have no block.
__device__ __forceinline__ int held_of(const Args &a, int length) {
  return static_cast<int>(min(static_cast<int64_t>(length), a.cols << a.log_b));
}

// Rows' results, from a wave: to the output, or to a split's part.
template <typename T, int D, int NQ>
__device__ __forceinline__ void store_rows(const Args &a, Wave<T, D, NQ> &w, int kvh, int first, int row0, int rows, int split) {
  const int lane = lane_id(), n = lane % 16, g = lane / 16, heads = a.kv_heads * a.group;
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    const int row = row0 + 16 * x + n;
    if (row >= rows) continue;
    const int64_t at = static_cast<int64_t>(first + row / a.group) * heads + kvh * a.group + row % a.group;
    const float inv = w.l[x] > 0.f ? 1.f / w.l[x] : (w.l[x] == 0.f ? 0.f : w.l[x]);  // a row that sees nothing: zeros
    const float f = inv * pow2(w.m2[x] - w.m[x]);
    if (a.part) {
      const int64_t to = static_cast<int64_t>(split) * a.tokens * heads + at;
      if (g == 0) a.part_ml[to] = make_float2(w.m[x], w.l[x]);
#pragma unroll
      for (int e = 0; e < w.ND; ++e) *reinterpret_cast<f4 *>(a.part + to * D + e * 16 + 4 * g) = w.acc[x][e] * f;
    } else {
      T *o = static_cast<T *>(a.out) + at * D;
      if (g == 0 && a.lse) a.lse[at] = lse_of(w.m[x], w.l[x]);
#pragma unroll
      for (int e = 0; e < w.ND; ++e) {
        T y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = static_cast<T>(w.acc[x][e][i] * f);
        __builtin_memcpy(__builtin_assume_aligned(o + e * 16 + 4 * g, 4 * sizeof(T)), y, sizeof(y));
      }
    }
  }
}

// Many rows: each of the four waves has 16 NQ of them and all walk the same
// tiles.  A tile is fetched and turned into f16 once per block, a quarter by
// each wave, into one of two LDS buffers: while a tile is worked on, the codes of
// the next are in flight to registers, and go to the other buffer between its two products.  No unit is
// full: VALU (softmax, conversion) 44% of the cycles (64% at D = 64), matrix cores 21 to 24%, waves waiting 31 to 35%; a
// wave's products, softmax and conversion follow one another, and two or three waves of a SIMD take turns.  The kernel alone: 8 requests of up to
// 2,048 new on up to 2,047 cached, causal, 16 heads of 128: 318 us, 580 TFLOP/s (668 us with every wave converting for
// itself); 64 x 1,024 candidates, 8 heads of 64: 271 us, 515 TFLOP/s.
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kWaves *kWave, D <= 128 ? 2 : 1) rows_kernel(Args a) {
  using W = Wave<T, D, NQ>;
  using R = RowTile<D>;
  constexpr int NT = kWaves * kWave, kPieces = 64 * D / 16 / NT;  // 16-byte pieces of keys (and of values) per thread
  static_assert(D >= 64, "a thread has a piece");
  __shared__ u4 buf[2][R::kKeys + R::kValues];
  const int tid = threadIdx.x, lane = lane_id(), g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  // With a causal mask, all requests' last rows first, since those see the most, turned by three from one row
  // tile to the next so that no XCD (blocks go to the eight in turn) has the same requests throughout; else every
  // row sees as much, and a request's rows come together, which finds its keys in the caches.  (8 requests x 2,048
  // causal: 365 us, 412 in the other order, 475 unturned; 64 x 1,024 candidates: 384 and 353.)
  const uint32_t pairs = a.requests * a.kv_heads, n = a.row_tiles * a.splits;
  const uint32_t place = a.causal ? blockIdx.x / pairs : blockIdx.x % n;
  const uint32_t pair = a.causal ? (blockIdx.x % pairs + 3 * place) % pairs : blockIdx.x / n;
  const int split = place % a.splits, rt = a.row_tiles - 1 - static_cast<int>(place / a.splits);
  const int kvh = pair % a.kv_heads, r = pair / a.kv_heads;
  const int first = a.cu[r], fresh = min(a.cu[r + 1], static_cast<int>(a.tokens)) - first;
  const int rows = min(fresh, a.max_q) * a.group;
  const int block_row0 = rt * kWaves * 16 * NQ, row0 = block_row0 + wave * 16 * NQ;
  if (first < 0 || fresh <= 0 || block_row0 >= rows) return;
  const int length = length_of(a, r), held = held_of(a, length);
  const int64_t split_lo = static_cast<int64_t>(split) * a.chunk;
  if (split > 0 && split_lo >= held) return;  // the combine knows that this split is empty

  W w;
  w.load_queries(a, r, kvh, min(row0, rows), rows, first, fresh, length);
  const int *table = a.table + r * a.cols;

  // positions that rows [b, e) see any of
  const auto span = [&](int b, int e, int &lo, int &hi) {
    lo = 0;
    hi = b < e ? held : 0;
    if (a.causal && b < e) {
      hi = min(held, max(0, length - fresh + (e - 1) / a.group + 1));
      if (a.window > 0) lo = first_seen(a, length - fresh + b / a.group);
    }
    if (a.part) {
      lo = max(lo, static_cast<int>(split_lo));
      hi = static_cast<int>(min(static_cast<int64_t>(hi), split_lo + a.chunk));
    }
  };
  int lo, hi, my_lo, my_hi;
  span(block_row0, min(block_row0 + kWaves * 16 * NQ, rows), lo, hi);
  span(row0, min(row0 + 16 * NQ, rows), my_lo, my_hi);
  const int tile_lo = lo / kTile, tile_hi = hi > lo ? (hi + kTile - 1) / kTile : 0;

  // A wave's pieces of one round (64 pieces of keys, 64 of values) lie in one chunk of 16 tokens, so block ids and
  // the chunk's addresses are scalars, and a thread's place in the chunk stays the same from tile to tile.  Key
  // pieces go to lanes so that eight lanes write their units to different banks: four of a token, four of the next.
  const int in_b = (1 << a.log_b) - 1;
  u4 kr[kPieces], vr[kPieces];
  const auto chunk_of = [&](int i) { return (i * NT + wave * kWave) / D; };
  constexpr int kHigh = D / 64;  // groups of four pieces of a token
  const auto token_of = [&](int i) { return (i * NT + tid) / (8 * kHigh) * 2 + (tid >> 2 & 1); };
  const auto part_of = [&](int i) { return (tid & 3) + (i * NT + tid) / 8 % kHigh * 4; };
  // the block of this lane's chunk; vector loads, since a scalar load would have every wait for LDS wait for it too
  const auto block_at = [&](int tile) { return block_of(a, table, tile * kTile + 16 * g); };
  const auto fetch = [&](int tile, int own) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int id = max(__builtin_amdgcn_readlane(own, 16 * chunk_of(i)), 0);
      const int64_t at = ((static_cast<int64_t>(id) * a.kv_heads + kvh) << (a.log_b - 4)) +
                         (((tile * kTile + 16 * chunk_of(i)) & in_b) >> 4);  // the chunk, of 16 D bytes
      const uint32_t ko = token_of(i) % 16 * D + part_of(i) * 16, vo = (i * NT + tid) % D * 16;
      kr[i] = *reinterpret_cast<const u4 *>(a.k + at * (16 * D) + ko);
      vr[i] = *reinterpret_cast<const u4 *>(a.v + at * (16 * D) + vo);
    }
  };
  const auto convert = [&](u4 *to) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int token = token_of(i), unit = part_of(i) * 2, t = token % 16 / 4, m = token / 16 * 4 + token % 4;
      to[R::key_at(t, m, unit)] = __builtin_bit_cast(u4, f16_of_codes(kr[i][0], kr[i][1]));
      to[R::key_at(t, m, unit + 1)] = __builtin_bit_cast(u4, f16_of_codes(kr[i][2], kr[i][3]));
      const int piece = i * NT + tid, chunk = piece / D, d = piece % D;
      to[R::kKeys + R::value_at(d, 2 * chunk)] = __builtin_bit_cast(u4, f16_of_codes(vr[i][0], vr[i][1]));
      to[R::kKeys + R::value_at(d, 2 * chunk + 1)] = __builtin_bit_cast(u4, f16_of_codes(vr[i][2], vr[i][3]));
    }
  };
  const auto scales = [&](int own, float &ks, float &vs) {
    const int64_t bh = static_cast<int64_t>(max(own, 0)) * a.kv_heads + kvh;
    ks = a.ks[bh];
    vs = a.vs[bh];
  };

  if (tile_lo < tile_hi) {
    int own = block_at(tile_lo), own1 = tile_lo + 1 < tile_hi ? block_at(tile_lo + 1) : -1, own2 = -1;
    float ks, vs, ks1 = 0.f, vs1 = 0.f;
    fetch(tile_lo, own);
    scales(own, ks, vs);
    convert(buf[0]);
    if (tile_lo + 1 < tile_hi) fetch(tile_lo + 1, own1);
    __syncthreads();
    for (int tile = tile_lo; tile < tile_hi; ++tile) {
      const u4 *now = buf[(tile - tile_lo) & 1];
      const bool more = tile + 1 < tile_hi;
      const bool mine = tile * kTile < my_hi && (tile + 1) * kTile > my_lo;
      if (more) scales(own1, ks1, vs1);
      if (tile + 2 < tile_hi) own2 = block_at(tile + 2);
      f4 s[NQ][4];
      if (mine) {
        w.scores(now, s);
        w.weights(s, ks, vs, own >= 0, tile * kTile);
      }
      if (more) convert(buf[(tile + 1 - tile_lo) & 1]);
      if (tile + 2 < tile_hi) fetch(tile + 2, own2);
      if (mine) w.values(now + R::kKeys, s);
      own = own1;
      own1 = own2;
      ks = ks1;
      vs = vs1;
      __syncthreads();
    }
  }
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    w.l[x] += xor16(w.l[x]);
    w.l[x] += xor32(w.l[x]);
  }
  store_rows(a, w, kvh, first, row0, rows, split);
}

// kKeys: the four waves of a block share its rows and take its tiles in turn; bound by the cache's bytes: 256
// requests x 66 to 8,192 tokens, 8 heads of 128: 2.17 GB in 400 us, 5.4 TB/s.
// (few rows, long histories); otherwise (D = 32) each wave has its own rows and all
// walk the same tiles.
template <typename T, int D, int NQ, bool kKeys>
__global__ void __launch_bounds__(kWaves *kWave) attention_kernel(Args a) {
  using W = Wave<T, D, NQ>;
  const int lane = lane_id(), wave = threadIdx.x / kWave, n = lane % 16, g = lane / 16;
  // all requests' parts in turn, so that the longest don't end alone
  const uint32_t pair = blockIdx.x % (a.requests * a.kv_heads), place = blockIdx.x / (a.requests * a.kv_heads);
  const int split = place % a.splits, rt = a.row_tiles - 1 - static_cast<int>(place / a.splits);
  const int kvh = pair % a.kv_heads, r = pair / a.kv_heads;
  const int first = a.cu[r], fresh = min(a.cu[r + 1], static_cast<int>(a.tokens)) - first;
  const int rows = min(fresh, a.max_q) * a.group;
  const int row0 = kKeys ? rt * 16 * NQ : (rt * kWaves + wave) * 16 * NQ;
  const int block_row0 = kKeys ? row0 : rt * kWaves * 16 * NQ;
  if (first < 0 || fresh <= 0 || block_row0 >= rows) return;
  const int length = length_of(a, r), held = held_of(a, length);
  const bool splits = a.part != nullptr;
  const int64_t split_lo = static_cast<int64_t>(split) * a.chunk;
  if (splits && split > 0 && split_lo >= held) return;  // the combine knows that this split is empty

  W w;
  w.load_queries(a, r, kvh, min(row0, rows), rows, first, fresh, length);
  const int *table = a.table + r * a.cols;

  // the tiles that any of the wave's rows sees
  int see_lo = 0x7fffffff, see_hi = 0;
#pragma unroll
  for (int x = 0; x < NQ; ++x)
    if (w.hi[x] > w.lo[x]) see_lo = min(see_lo, w.lo[x]), see_hi = max(see_hi, w.hi[x]);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    see_lo = min(see_lo, __shfl_xor(see_lo, o));
    see_hi = max(see_hi, __shfl_xor(see_hi, o));
  }
  see_lo = __builtin_amdgcn_readfirstlane(see_lo);
  see_hi = min(__builtin_amdgcn_readfirstlane(see_hi), held);
  if (splits) {
    see_lo = max(see_lo, static_cast<int>(min(split_lo, int64_t(0x7fffffff))));
    see_hi = static_cast<int>(min(static_cast<int64_t>(see_hi), split_lo + a.chunk));
  }
  const int tile_lo = see_lo / kTile, tile_hi = see_hi > see_lo ? (see_hi + kTile - 1) / kTile : 0;
  // Loads run ahead of the products: a tile's keys are fetched while the tile before it is weighted, its values and
  // scales while the tile before it ends, its block ids one tile earlier still.
  const int step = kKeys ? kWaves : 1;
  int tile = tile_lo + (kKeys ? wave : 0);
  if (tile < tile_hi) {
    Ids now = ids_of(a, table, tile), next = tile + step < tile_hi ? ids_of(a, table, tile + step) : Ids{-1, -1};
    u4 kr[4][W::NK], vr[W::ND];
    float ks, vs;
    load_keys<D>(a, now, kvh, tile, kr);
    load_values<D>(a, now, kvh, tile, vr, ks, vs);
    while (true) {
      const int base = tile * kTile;
      const bool more = tile + step < tile_hi, ok = now.own >= 0;
      f4 s[NQ][4];
      w.scores(kr, s);
      now = next;
      if (more) {
        load_keys<D>(a, next, kvh, tile + step, kr);
        if (tile + 2 * step < tile_hi) next = ids_of(a, table, tile + 2 * step);
      }
      w.weights(s, ks, vs, ok, base);
      w.values(vr, s);
      if (!more) break;
      tile += step;
      load_values<D>(a, now, kvh, tile, vr, ks, vs);
    }
  }

  // join the lane groups' sums; then, for kKeys, the waves
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    w.l[x] += xor16(w.l[x]);
    w.l[x] += xor32(w.l[x]);
  }
  __shared__ float jm[kWaves][16 * NQ], jm2[kWaves][16 * NQ], jl[kWaves][16 * NQ];
  __shared__ float ja[kKeys ? 2 : 1][kKeys ? 16 * NQ * (D + 4) : 1];
  if constexpr (kKeys) {
#pragma unroll
    for (int x = 0; x < NQ; ++x)
      if (g == 0) jm[wave][x * 16 + n] = w.m[x], jm2[wave][x * 16 + n] = w.m2[x];
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
      float top = kNone, top2 = kNone;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) top = fmaxf(top, jm[k][x * 16 + n]), top2 = fmaxf(top2, jm2[k][x * 16 + n]);
      const float by = pow2(w.m2[x] - top2);
      w.l[x] *= pow2(w.m[x] - top);
      w.m[x] = top;
      w.m2[x] = top2;
#pragma unroll
      for (int e = 0; e < W::ND; ++e) w.acc[x][e] *= by;
      if (g == 0) jl[wave][x * 16 + n] = w.l[x];
    }
    // waves 2, 3 into 0, 1, then 1 into 0
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
      if (wave >= half && wave < 2 * half)
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
          for (int e = 0; e < W::ND; ++e)
            *reinterpret_cast<f4 *>(&ja[wave - half][(x * 16 + n) * (D + 4) + e * 16 + 4 * g]) = w.acc[x][e];
      __syncthreads();
      if (wave < half)
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
          for (int e = 0; e < W::ND; ++e)
            w.acc[x][e] += *reinterpret_cast<const f4 *>(&ja[wave][(x * 16 + n) * (D + 4) + e * 16 + 4 * g]);
      __syncthreads();
    }
    if (wave > 0) return;
#pragma unroll
    for (int x = 0; x < NQ; ++x) w.l[x] = jl[0][x * 16 + n] + jl[1][x * 16 + n] + jl[2][x * 16 + n] + jl[3][x * 16 + n];
  }

  store_rows(a, w, kvh, first, row0, rows, split);
}

// Joins the splits of each (token, head), one block per row: the threads' first
// pass finds the largest maximum, then each of 1024 / D groups of D / 4
// threads adds every such group's share of the splits, four elements a thread.
template <typename T, int D>
__global__ void __launch_bounds__(256) combine_kernel(Args a, int requests, int64_t first_row) {
  constexpr int kPer = D / 4, kGroups = 256 / kPer;
  const int heads = a.kv_heads * a.group, tid = threadIdx.x;
  const int64_t row = first_row + blockIdx.x;
  const int tok = static_cast<int>(row / heads);
  int lo = 0, hi = requests;  // the last request that begins at or before tok
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= tok)
      lo = mid;
    else
      hi = mid;
  }
  if (tok < a.cu[lo] || tok >= a.cu[lo + 1]) return;
  if (tok - a.cu[lo] >= a.max_q) return;
  const int n = max(1, static_cast<int>((static_cast<int64_t>(held_of(a, length_of(a, lo))) + a.chunk - 1) / a.chunk));
  const int64_t step = a.tokens * heads;
  __shared__ float wave_top[4], weight[256];
  __shared__ f4 joined[kGroups][kPer];
  float top = kNone;
  for (int i = tid; i < n; i += 256) top = fmaxf(top, a.part_ml[i * step + row].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  if (lane_id() == 0) wave_top[tid / kWave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
  const int mine = tid / kPer, at = tid % kPer;
  const f4 *part = reinterpret_cast<const f4 *>(a.part) + row * kPer + at;
  f4 o = {0.f, 0.f, 0.f, 0.f};
  float total = 0.f;
  for (int base = 0; base < n; base += 256) {
    const int held = min(n - base, 256);
    if (base > 0) __syncthreads();
    if (tid < held) {
      const float2 ml = a.part_ml[(base + tid) * step + row];
      weight[tid] = __builtin_amdgcn_exp2f(ml.x - top) * ml.y;
    }
    __syncthreads();
#pragma unroll 4
    for (int i = mine; i < held; i += kGroups) {
      const float w = weight[i];
      const f4 y = part[(base + i) * step * kPer];
      total += w;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __builtin_fmaf(w, y[j], o[j]);
    }
  }
  __shared__ float totals[kGroups];
  joined[mine][at] = o;
  if (at == 0) totals[mine] = total;
  __syncthreads();
  if (mine > 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k) {
    o += joined[k][at];
    total += totals[k];
  }
  const float inv = total > 0.f ? 1.f / total : total;  // no split sees anything: zeros
  T *out = static_cast<T *>(a.out) + row * D + at * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) out[j] = static_cast<T>(o[j] * inv);
  if (at == 0 && a.lse) a.lse[row] = lse_of(top, total);
}

struct Plan {
  bool keys;
  int nq, row_tiles, splits, chunk;
};

// 16-row tiles of a wave where it has rows of its own.
constexpr int row_tiles_of(int dim) { return dim == 256 ? 1 : 2; }

Plan plan(int64_t requests, int64_t kv_heads, int64_t group, int64_t dim, int64_t max_q, int64_t max_len) {
  Plan p{};
  const int64_t rows = max_q * group;
  // Keys shared by a block's waves: for one tile of rows; and for up to 64 rows (in tiles of 32) of long histories,
  // where waves with rows of their own would mostly have none (64 requests x up to 4,096, 4 heads of 128: 32 rows 70 us
  // against 94, 64 rows 97 against 109; 2 heads of 64, 24 rows: 33 against 61).  Not for short ones (256 requests x
  // 300: 49 against 34, the join weighs more than the tiles) nor for D = 256 (56 against 55).
  p.keys = rows <= 16 || (rows <= 64 && dim <= 128 && max_len >= 1024);
  p.nq = !p.keys ? row_tiles_of(static_cast<int>(dim)) : rows <= 16 ? 1 : 2;
  const int64_t per = p.keys ? 16 * p.nq : 16 * p.nq * kWaves;
  p.row_tiles = static_cast<int>((rows + per - 1) / per);
  const int64_t blocks = requests * kv_heads * p.row_tiles;
  const int64_t most = (max_len + 255) / 256;
  // With keys shared by a block's waves: two blocks per CU, or four of the smaller dims (more splits cost a join
  // and a part each: 64 requests x 2,048, 8 heads of 128 take 37 us in one split, 43 in two, 50 in eight; 64 x 8,192, 4
  // heads of 64 take 45, 36 and 41 in two, four and sixteen), none for fewer than 256 tokens, and one launch
  // up to 1,024 (the GPU takes 1 us longer, the host 3 us less).  With rows of their own: only where the rows
  // leave most of the GPU idle.
  const int64_t want = p.keys && dim <= 64 ? 1024 : 512;
  int64_t s = blocks > 0 ? (want + blocks - 1) / blocks : 1;
  if (p.keys ? max_len <= 1024 : blocks > 256) s = 1;
  if (s > most) s = most;
  if (s < 1) s = 1;
  int64_t chunk = (max_len + s - 1) / s;
  chunk = (chunk + 255) / 256 * 256;
  if (chunk < 256) chunk = 256;
  p.splits = static_cast<int>(max_len > 0 ? (max_len + chunk - 1) / chunk : 1);
  p.chunk = static_cast<int>(chunk);
  return p;
}

template <typename T, int D>
void launch_requests(const Args &a, const Plan &p, unsigned grid, hipStream_t stream) {
  if (p.keys && p.nq == 1) {
    attention_kernel<T, D, 1, true><<<grid, kWaves * kWave, 0, stream>>>(a);
  } else if (p.keys) {
    if constexpr (D <= 128) attention_kernel<T, D, 2, true><<<grid, kWaves * kWave, 0, stream>>>(a);
  } else if constexpr (D == 32)
    attention_kernel<T, D, row_tiles_of(D), false><<<grid, kWaves * kWave, 0, stream>>>(a);
  else
    rows_kernel<T, D, row_tiles_of(D)><<<grid, kWaves * kWave, 0, stream>>>(a);
}

template <typename T, int D>
hlr_status launch(const Args &a, const Plan &p, int64_t requests, hipStream_t stream) {
  const int64_t each = static_cast<int64_t>(p.splits) * p.row_tiles * a.kv_heads, most = most_blocks(kWaves * kWave) / each;
  for (int64_t r = 0; r < requests; r += most) {
    Args b = a;
    b.table += r * a.cols;
    b.lengths += r;
    b.cu += r;
    b.requests = static_cast<uint32_t>(requests - r < most ? requests - r : most);
    launch_requests<T, D>(b, p, static_cast<unsigned>(each * b.requests), stream);
    const hlr_status st = launch_status();
    if (st != HLR_OK) return st;
  }
  if (p.splits > 1) {
    const int64_t rows = a.tokens * a.kv_heads * a.group;
    for (int64_t r = 0; r < rows; r += most_blocks(256)) {
      const int64_t here = rows - r < most_blocks(256) ? rows - r : most_blocks(256);
      combine_kernel<T, D><<<static_cast<unsigned>(here), 256, 0, stream>>>(a, static_cast<int>(requests), r);
      const hlr_status st = launch_status();
      if (st != HLR_OK) return st;
    }
  }
  return HLR_OK;
}

template <typename T>
hlr_status launch_dim(const Args &a, const Plan &p, int64_t dim, int64_t requests, hipStream_t stream) {
  switch (dim) {
    case 32: return launch<T, 32>(a, p, requests, stream);
    case 64: return launch<T, 64>(a, p, requests, stream);
    case 128: return launch<T, 128>(a, p, requests, stream);
    default: return launch<T, 256>(a, p, requests, stream);
  }
}

bool sizes_ok(int64_t tokens, int64_t requests, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t max_q,
              int64_t max_len) {
  return tokens >= 0 && requests >= 0 && requests <= HLR_HIST_MAX_REQUESTS && kv_heads > 0 && kv_heads <= 65535 &&
         q_heads >= kv_heads && q_heads % kv_heads == 0 && q_heads <= 65535 && tokens <= kMaxN / q_heads && max_q >= 0 &&
         max_q <= kMaxN / q_heads && max_len >= 0 && max_len <= kMaxN - 65536 &&
         (dim == 32 || dim == 64 || dim == 128 || dim == 256);
}

}  // namespace

extern "C" size_t hist_attention_workspace_size(int64_t tokens, int64_t requests, int64_t q_heads, int64_t kv_heads,
                                                int64_t dim, int64_t max_q, int64_t max_len) {
  if (!sizes_ok(tokens, requests, q_heads, kv_heads, dim, max_q, max_len)) return 0;
  const Plan p = plan(requests, kv_heads, q_heads / kv_heads, dim, max_q, max_len);
  if (p.splits <= 1) return 0;
  const size_t rows = static_cast<size_t>(p.splits) * tokens * q_heads;
  return round_up(rows * dim * 4, 256) + round_up(rows * 8, 256);
}

extern "C" hlr_status hist_attention(const void *q, int32_t type, int64_t tokens, int64_t q_heads, int64_t q_token_stride,
                                     int64_t q_head_stride, const int8_t *k_codes, const int8_t *v_codes,
                                     const float *k_scale, const float *v_scale, int64_t num_blocks, int64_t kv_heads,
                                     int64_t block, int64_t dim, const int32_t *block_table, int64_t table_cols,
                                     const int32_t *lengths, const int32_t *cu, int64_t requests, int64_t max_q,
                                     int64_t max_len, float scale, int32_t causal, int64_t window, void *out,
                                     float *out_lse, void *ws, size_t ws_bytes, hipStream_t stream) {
  if (dim != 32 && dim != 64 && dim != 128 && dim != 256) return HLR_UNSUPPORTED_DIM;
  if (!sizes_ok(tokens, requests, q_heads, kv_heads, dim, max_q, max_len) || type < 0 || type > 2 ||
      (causal != 0 && causal != 1) || window < 0 || window > kMaxN || (window > 0 && !causal) || num_blocks < 0 ||
      num_blocks > kMaxN || table_cols < 0 || table_cols > kMaxN / 256 || !(scale == scale))
    return HLR_INVALID_ARG;
  int log_b = 4;
  while (log_b <= 8 && (int64_t(1) << log_b) != block) ++log_b;
  if (log_b > 8) return HLR_INVALID_ARG;
  if (tokens == 0 || requests == 0 || max_q == 0) return HLR_OK;
  if (!q || !out || !lengths || !cu || (table_cols > 0 && !block_table) ||
      (num_blocks > 0 && (!k_codes || !v_codes || !k_scale || !v_scale)))
    return HLR_INVALID_ARG;
  const int64_t unit = type == HLR_FP32 ? 4 : 8;
  if (!aligned(q, 16) || !aligned(out, 16) || q_token_stride % unit || q_head_stride % unit || !aligned(k_codes, 16) ||
      !aligned(v_codes, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) ||
      !aligned(lengths, 4) || !aligned(cu, 4) || !aligned(out_lse, 4))
    return HLR_MISALIGNED;
  const Plan p = plan(requests, kv_heads, q_heads / kv_heads, dim, max_q, max_len);
  if (static_cast<int64_t>(p.splits) * p.row_tiles > most_blocks(kWaves * kWave) / kv_heads) return HLR_INVALID_ARG;
  Args a{};
  a.q = q;
  a.q_tok = q_token_stride;
  a.q_head = q_head_stride;
  a.k = k_codes;
  a.v = v_codes;
  a.ks = k_scale;
  a.vs = v_scale;
  a.table = block_table;
  a.cols = num_blocks > 0 ? table_cols : 0;  // no pool: every request sees nothing
  a.lengths = lengths;
  a.cu = cu;
  a.out = out;
  a.lse = out_lse;
  a.tokens = tokens;
  a.num_blocks = num_blocks;
  a.kv_heads = static_cast<int>(kv_heads);
  a.group = static_cast<int>(q_heads / kv_heads);
  a.log_b = log_b;
  a.causal = causal;
  a.window = static_cast<int>(window);
  a.scale = scale * 1.44269504088896340736f;
  a.chunk = p.chunk;
  a.row_tiles = p.row_tiles;
  a.splits = static_cast<uint32_t>(p.splits);
  a.max_q = static_cast<int>(max_q);
  a.max_len = static_cast<int>(max_len);
  if (p.splits > 1) {
    const size_t need = hist_attention_workspace_size(tokens, requests, q_heads, kv_heads, dim, max_q, max_len);
    if (!ws || ws_bytes < need) return HLR_WORKSPACE_TOO_SMALL;
    if (!aligned(ws, 256)) return HLR_MISALIGNED;
    Carver c(ws);
    a.part = c.take<float>(static_cast<size_t>(p.splits) * tokens * q_heads * dim);
    a.part_ml = c.take<float2>(static_cast<size_t>(p.splits) * tokens * q_heads);
  }
  if (type == HLR_FP32) return launch_dim<float>(a, p, dim, requests, stream);
  if (type == HLR_BF16) return launch_dim<bf16>(a, p, dim, requests, stream);
  return launch_dim<_Float16>(a, p, dim, requests, stream);
}
