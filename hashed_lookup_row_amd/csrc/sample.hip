// Sampling one item per row of scores with temperature, top-k, top-p and
// min-p, from given random numbers.
//
// With f = log2(e) / temperature, w = 2^((x - max x) f); items rank by (x
// descending, index ascending); the filters keep a prefix of that order:
//   top-k  the first k
//   top-p  item i while the mass (sum of w) of the items before it is below
//          top_p times the mass of the first k
//   min-p  w >= min_p
// and always the first item.  Of the kept items the one with the largest
// x / temperature - log(noise) is drawn (noise ~ Exp(1): an exponential race, so
// item i wins with probability w_i over the kept mass).  Only the kept items'
// noise is read.
//
// One block per row:
//   1. the maximum, each thread's own maximum, and the sum of w (against a
//      running maximum per thread);
//   2. a bound below which no kept item lies: min-p's own, and the r-th largest
//      of the threads' maxima (at least r items reach it), r = k, or half
//      the threads where top-k is off.  The items that reach it, about as many
//      as r, go to a list in LDS;
//   3. a list of at most one item per thread is sorted by (x, index), and rank,
//      mass before and the race follow per thread.
// Where the list doesn't hold the prefix or is too long (a flat row with a
// large top-p, many equal scores), the prefix is found as a threshold over the
// list or the row itself, by counts for top-k and by masses for top-p: linear
// bins of log2 w and a sort of the edge's bin (find_edge; select_share for
// top-p alone over a row), or where that bin holds too many items a radix
// selection (select_prefix).  Masses are whole numbers in units of the
// total's 2^-31, so that no result hangs on the order of atomics; top-p's share
// is taken of their own sum.  Half a unit for each of n items is n 2^-32 of the
// total, by which a share's edge may be off at the most: 3e-5 for 131,072 items.
//
// Measured: 256 x 1,024 fp32 12 us (a sort of 1,024 per CU); 256 x 131,072
// bf16 39 us with top-k 50 (14 us the first reading, 15 the second, from the
// caches), 106 to 133 with top-p alone (two passes more, their items' masses,
// bins and races), 65 without a filter (scores and noise once); one row of
// 32,003 fp32 20 us (latency).  For rows over 8,192 items the rare paths' code takes the
// kernel to its 128 registers, with 53 to 57 of them spilled.
#include "hlr_common.hpp"
#include "hist_common.hpp"

#include <type_traits>

namespace {
using namespace hlr;

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr float kUnits = 2147483648.f;  // 2^31
constexpr int kBins = 2048;
constexpr int kList = 6144;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kMost = 3.402823466e38f;

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);  // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __builtin_bit_cast(float, (k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// NaN counts as -inf, +inf as the largest number.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -__builtin_inff()), kMost); }
// The key of an item: 0 for those that can't be drawn.
__device__ __forceinline__ uint32_t item_key(float x) { return x > -__builtin_inff() ? key_of(x) : 0u; }

struct SampleArgs {
  const void *scores;
  int64_t stride;
  const float *noise;
  int64_t noise_stride;
  const float *temperature;
  const int *top_k;
  const float *top_p, *min_p;
  int64_t items;
  int64_t *index;
  float *logprob;
  int64_t first;  // row of this launch's first block
};

// What a row's items are measured against.
struct Scale {
  float top, f;  // the largest x; log2(e) / temperature
  float units;   // of mass per weight: 2^31 over a bound of the weights that are added up
  __device__ __forceinline__ float weight(float x) const { return __builtin_amdgcn_exp2f((x - top) * f); }
  __device__ __forceinline__ uint32_t mass(float x) const { return static_cast<uint32_t>(weight(x) * units + 0.5f); }
};

// A granule: 16 bytes of scores, of any alignment.
template <typename T>
struct Granule {
  static constexpr int N = 16 / sizeof(T);
  u4 raw;
  static constexpr uint64_t kInf = sizeof(T) == 4                ? 0xff800000ff800000ull
                                   : std::is_same<T, bf16>::value ? 0xff80ff80ff80ff80ull
                                                                  : 0xfc00fc00fc00fc00ull;  // -inf, repeated
  // A granule that lies in the row; -inf for others.
  __device__ __forceinline__ void load(const T *x, int first, int items) {
    const uint64_t none[2] = {kInf, kInf};
    __builtin_memcpy(&raw, none, 16);
    if (first <= items - N) __builtin_memcpy(&raw, x + first, 16);
  }
  // The granule that a row of at least one granule ends in: its last 16 bytes moved down, -inf past them.
  __device__ __forceinline__ void load_end(const T *x, int first, int items) {
    uint64_t w[2] = {kInf, kInf};
    if (first < items) {
      const int bits = (first + N - items) * static_cast<int>(8 * sizeof(T));
      __builtin_memcpy(w, x + items - N, 16);
      if (bits < 64) {
        w[0] = w[0] >> bits | w[1] << (64 - bits);
        w[1] = w[1] >> bits | kInf << (64 - bits);
      } else {
        w[0] = bits == 64 ? w[1] : w[1] >> (bits - 64) | kInf << (128 - bits);
        w[1] = kInf;
      }
    }
    __builtin_memcpy(&raw, w, 16);
  }
  __device__ __forceinline__ float at(int j) const {
    T t[N];
    __builtin_memcpy(t, &raw, 16);
    return clean(static_cast<float>(t[j]));
  }
};

// The whole row, from memory, two granules in flight per thread (four take as long or longer).
template <typename T, int NT>
struct RowItems {
  using G = Granule<T>;
  const T *x;
  int items;
  template <typename F>
  __device__ __forceinline__ void each_granule(F f) const {
    constexpr int kAhead = 2;
#pragma unroll 1
    for (int first = threadIdx.x * G::N; first < items; first += kAhead * NT * G::N) {
      G g[kAhead];
#pragma unroll
      for (int v = 0; v < kAhead; ++v) g[v].load(x, first + v * NT * G::N, items);
#pragma unroll
      for (int v = 0; v < kAhead; ++v) f(first + v * NT * G::N, g[v]);
    }
    const int end = items / G::N * G::N;  // the granule the row ends in, if it ends within one, is one thread's
    if (threadIdx.x == NT - 1 && end < items) {
      G g;
      g.load_end(x, end, items);
      f(end, g);
    }
  }
  // Scores: -inf for items that can't be drawn.
  template <typename F>
  __device__ __forceinline__ void each_score(F f) const {
    each_granule([&](int first, const G &g) {
#pragma unroll
      for (int j = 0; j < G::N; ++j) f(first + j, g.at(j));
    });
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each_score([&](int i, float y) { f(i, item_key(y)); });
  }
};

// The list in LDS: key and complemented index.
template <int NT>
struct ListItems {
  const uint64_t *list;
  int n;
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int i = threadIdx.x; i < n; i += NT) {
      const uint64_t c = list[i];
      f(static_cast<int>(~static_cast<uint32_t>(c)), static_cast<uint32_t>(c >> 32));
    }
  }
};

// Items as another function enumerates them.
template <typename Each>
struct Through {
  const Each &by;
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    by(f);
  }
};

// ---- reductions over a block; tmp holds 17 entries
template <int NT>
__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t *tmp) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint64_t y = __shfl_xor(v, o);
    v = y > v ? y : v;
  }
  __syncthreads();
  if (lane_id() == 0) tmp[threadIdx.x / kWave] = v;
  __syncthreads();
  v = tmp[0];
#pragma unroll
  for (int w = 1; w < NT / kWave; ++w) v = tmp[w] > v ? tmp[w] : v;
  return v;
}

template <int NT>
__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t *tmp) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if (lane_id() == 0) tmp[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w) v += tmp[w];
  return v;
}

template <int NT>
__device__ __forceinline__ float block_sum(float v, uint64_t *tmp) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  float *t = reinterpret_cast<float *>(tmp);
  __syncthreads();
  if (lane_id() == 0) t[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w) v += t[w];
  return v;
}

// The value of lane ^ J, without LDS.
template <int J>
__device__ __forceinline__ uint32_t from_lane_xor(uint32_t v) {
  const int x = static_cast<int>(v);
  if constexpr (J == 1) {
    return __builtin_amdgcn_mov_dpp(x, 0xB1, 0xf, 0xf, true);  // quad_perm 1 0 3 2
  } else if constexpr (J == 2) {
    return __builtin_amdgcn_mov_dpp(x, 0x4E, 0xf, 0xf, true);  // quad_perm 2 3 0 1
  } else if constexpr (J == 4) {  // row_half_mirror (lane ^ 7), then quad_perm 3 2 1 0 (lane ^ 3)
    return __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(x, 0x141, 0xf, 0xf, true), 0x1B, 0xf, 0xf, true);
  } else if constexpr (J == 8) {
    return __builtin_amdgcn_mov_dpp(x, 0x128, 0xf, 0xf, true);  // row_ror 8
  } else if constexpr (J == 16) {
    const auto y = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (lane_id() & 16) ? y[0] : y[1];
  } else {
    const auto y = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (lane_id() & 32) ? y[0] : y[1];
  }
}
template <int J>
__device__ __forceinline__ uint64_t from_lane_xor(uint64_t v) {
  return static_cast<uint64_t>(from_lane_xor<J>(static_cast<uint32_t>(v >> 32))) << 32 |
         from_lane_xor<J>(static_cast<uint32_t>(v));
}

// The lanes whose bit J is clear (J below 64).
constexpr uint64_t lanes_without(int J) {
  uint64_t m = 0;
  for (int i = 0; i < kWave; ++i)
    if ((i & J) == 0) m |= 1ull << i;
  return m;
}
// One step of the bitonic network: the larger of v and y goes to the thread
// whose bits J and K are alike.  In a wave those are lanes known at compile
// time, all or none of them flipped where K is a bit of the wave's number.
template <int K, int J, typename U>
__device__ __forceinline__ U keep(U v, U y) {
  bool larger;
  if constexpr (J < kWave && K < kWave)
    larger = __builtin_amdgcn_inverse_ballot_w64(~(lanes_without(J) ^ lanes_without(K)));
  else {
    const bool k = (__builtin_amdgcn_readfirstlane(threadIdx.x) & K) == 0;
    if constexpr (J < kWave)
      larger = __builtin_amdgcn_inverse_ballot_w64(k ? lanes_without(J) : ~lanes_without(J));
    else
      larger = ((__builtin_amdgcn_readfirstlane(threadIdx.x) & J) == 0) == k;
  }
  return (v > y) == larger ? v : y;
}
template <int K, int J, typename U>
__device__ __forceinline__ U merge_in_wave(U v) {
  v = keep<K, J>(v, from_lane_xor<J>(v));
  if constexpr (J > 1) v = merge_in_wave<K, J / 2>(v);
  return v;
}
template <int NT, int K, int J, typename U>
__device__ __forceinline__ U merge(U v, bool counts, U *buf, int &turn) {
  if constexpr (J >= kWave) {
    U *b = buf + (turn ^= 1) * NT;  // the buffers take turns, so one barrier per step is enough
    if (counts) b[threadIdx.x] = v;
    __syncthreads();
    if (counts) v = keep<K, J>(v, b[threadIdx.x ^ J]);
    return merge<NT, K, J / 2>(v, counts, buf, turn);
  } else {
    return counts ? merge_in_wave<K, J>(v) : v;
  }
}
template <int NT, int K, typename U>
__device__ __forceinline__ U sort_from(U v, int size, bool counts, U *buf, int &turn) {
  if (K > size) return v;
  v = merge<NT, K, K / 2>(v, counts, buf, turn);
  if constexpr (K < NT) v = sort_from<NT, 2 * K>(v, size, counts, buf, turn);
  return v;
}
// The sum of the threads before this one.
template <int NT>
__device__ __forceinline__ uint64_t block_before(uint64_t v, uint64_t *tmp) {
  uint64_t run = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint64_t y = __shfl_up(run, o);
    if (lane_id() >= o) run += y;
  }
  __syncthreads();
  if (lane_id() == kWave - 1) tmp[threadIdx.x / kWave] = run;
  __syncthreads();
  run -= v;
  for (int w = 0; w < static_cast<int>(threadIdx.x) / kWave; ++w) run += tmp[w];
  return run;
}

// Sorts one value per thread of the first `size` threads (a power of two from
// 64) in descending order by the bitonic network; buf holds 2 NT.
template <int NT, typename U>
__device__ __forceinline__ U block_sort(U v, int size, U *buf) {
  int turn = 0;
  __syncthreads();
  return sort_from<NT, 2>(v, size, static_cast<int>(threadIdx.x) < size, buf, turn);
}

// Finds, among the items with key >= floor, the lowest key t above which the
// total is still below `target`; `above` receives the total above t.  Totals are
// counts (kMassed false) or masses.
template <bool kMassed, int NT, typename Items>
__device__ uint32_t select_key(const Items &items, uint32_t floor, Scale sc, uint64_t target, uint64_t *buf,
                               uint64_t *tmp, uint64_t &above) {
  uint32_t *bins = reinterpret_cast<uint32_t *>(buf);
  uint32_t prefix = 0, mask = 0;
  above = 0;
  const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = shifts[pass];
    const uint32_t field = (1u << widths[pass]) - 1u;
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += NT) bins[i] = 0;
    __syncthreads();
    items.each([&](int, uint32_t k) {
      if (k != 0 && k >= floor && (k & mask) == prefix)
        atomicAdd(&bins[(k >> shift) & field], kMassed ? sc.mass(of_key(k)) : 1u);
    });
    __syncthreads();
    // bins descend in rank; the last non-empty one whose total above is below the target
    constexpr int per = kBins / NT;
    uint64_t mine = 0;
    const int b0 = kBins - 1 - threadIdx.x * per;
#pragma unroll
    for (int j = 0; j < per; ++j) mine += bins[b0 - j];
    uint64_t incl = mine;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const uint64_t y = __shfl_up(incl, o);
      if (lane_id() >= o) incl += y;
    }
    __syncthreads();
    if (lane_id() == kWave - 1) tmp[threadIdx.x / kWave] = incl;
    __syncthreads();
    uint64_t run = above + incl - mine;
    for (int w = 0; w < static_cast<int>(threadIdx.x) / kWave; ++w) run += tmp[w];
    int best = -1;
    uint64_t best_above = 0;
#pragma unroll
    for (int j = 0; j < per; ++j) {
      const uint32_t c = bins[b0 - j];
      if (c != 0 && run < target) best = kBins - 1 - (b0 - j), best_above = run;
      run += c;
    }
    const uint32_t win = static_cast<uint32_t>(block_max<NT>(static_cast<uint64_t>(best + 1), tmp));
    if (win == 0) return 0;  // nothing there
    if (static_cast<uint32_t>(best + 1) == win) tmp[16] = best_above;
    __syncthreads();
    above = tmp[16];
    prefix |= (kBins - win) << shift;
    mask |= field << shift;
  }
  return prefix;
}

struct Filters {
  int k;         // 0: none
  float p, min;  // 1, 0: none
};

struct Drawn {
  uint32_t key, index;
};

// The race, for items in any order: by score, then by rank.
struct Race {
  float score = -__builtin_inff();
  uint32_t key = 0, index = 0;  // key 0: nobody yet
  __device__ __forceinline__ void enter(float s, uint32_t k, uint32_t i) {
    if (s == s && (key == 0 || s > score || (s == score && (k > key || (k == key && i < index))))) score = s, key = k, index = i;
  }
  __device__ __forceinline__ void meet(const Race &y) {
    if (y.key != 0) enter(y.score, y.key, y.index);
  }
  template <int NT>
  __device__ __forceinline__ void block_join(uint64_t *buf) {  // 2 * NT / 64 entries
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      Race y;
      y.score = __shfl_xor(score, o);
      y.key = static_cast<uint32_t>(__shfl_xor(static_cast<int>(key), o));
      y.index = static_cast<uint32_t>(__shfl_xor(static_cast<int>(index), o));
      meet(y);
    }
    __syncthreads();
    if (lane_id() == 0) {
      buf[threadIdx.x / kWave] = static_cast<uint64_t>(key) << 32 | index;
      buf[NT / kWave + threadIdx.x / kWave] = __builtin_bit_cast(uint32_t, score);
    }
    __syncthreads();
    for (int w = 0; w < NT / kWave; ++w) {
      Race y;
      y.score = __builtin_bit_cast(float, static_cast<uint32_t>(buf[NT / kWave + w]));
      y.key = static_cast<uint32_t>(buf[w] >> 32);
      y.index = static_cast<uint32_t>(buf[w]);
      meet(y);
    }
  }
};

// top-p's share of a mass; at least 1, so that the first item stays.
__device__ __forceinline__ uint64_t share_of(uint64_t total, float p) {
  const double want = static_cast<double>(p) * static_cast<double>(total);
  return want > 1.0 ? static_cast<uint64_t>(want) : 1;
}

// The kept prefix as a threshold, over items in any order.  all: the items are
// the whole row (else, without top-k, the row's mass is 2^31 units).
template <int NT, typename Items>
__device__ Drawn select_prefix(const Items &items, Scale sc, Filters flt, float divisor, const float *noise,
                               bool all, uint64_t *bins, uint64_t *tmp) {
  uint32_t edge = 1;  // kept: keys above `edge`, and of those equal to it the first `ties` by index
  uint64_t ties = ~0ull, above;
  if (flt.k > 0) {
    const uint32_t t = select_key<false, NT>(items, 1, sc, static_cast<uint64_t>(flt.k), bins, tmp, above);
    edge = t;
    ties = static_cast<uint64_t>(flt.k) - above;
  }
  if (flt.p < 1.f) {
    // the mass above the edge, and with `ties` of the items at it (or all, if fewer)
    uint64_t above_edge = 0, at_edge = 0;
    items.each([&](int, uint32_t q) {
      if (q > edge) above_edge += sc.mass(of_key(q));
      if (q == edge) ++at_edge;
    });
    above_edge = block_sum<NT>(above_edge, tmp);
    at_edge = block_sum<NT>(at_edge, tmp);
    const uint64_t w = flt.k > 0 ? sc.mass(of_key(edge)) : 0;
    uint64_t total = above_edge + (at_edge < ties ? at_edge : ties) * w;
    if (flt.k == 0 && !all) total = static_cast<uint64_t>(kUnits);
    const uint64_t goal = share_of(total, flt.p);
    if (flt.k > 0 && above_edge < goal) {
      const uint64_t n = w > 0 ? (goal - above_edge + w - 1) / w : ~0ull;
      ties = n < ties ? n : ties;
    } else {
      const uint32_t t = select_key<true, NT>(items, edge + 1, sc, goal, bins, tmp, above);
      if (t != 0) {
        const uint64_t wt = sc.mass(of_key(t));
        ties = wt > 0 ? (goal - above + wt - 1) / wt : ~0ull;
        edge = t;
      }
    }
  }
  // the first item, and how many are equal to the edge
  const uint32_t best = key_of(sc.top);
  uint32_t first = 0xffffffffu;
  uint64_t equal = 0;
  items.each([&](int i, uint32_t q) {
    if (q == best) first = min(first, static_cast<uint32_t>(i));
    equal += q == edge;
  });
  first = ~static_cast<uint32_t>(block_max<NT>(static_cast<uint64_t>(~first), tmp));
  equal = block_sum<NT>(equal, tmp);
  uint32_t last = 0xffffffffu;  // the last index kept of the items at the edge
  if (equal > ties) {
    // the ties-th of them: their complemented indexes as keys
    const auto by_index = [&](auto f) { items.each([&](int i, uint32_t q) { f(i, q == edge ? ~static_cast<uint32_t>(i) : 0u); }); };
    last = ~select_key<false, NT>(Through<decltype(by_index)>{by_index}, 1, sc, ties, bins, tmp, above);
  }
  Race race;
  items.each([&](int i, uint32_t q) {
    if (q == 0 || q < edge) return;
    if (q == edge && static_cast<uint32_t>(i) > last) return;
    if (!(sc.weight(of_key(q)) >= flt.min) && static_cast<uint32_t>(i) != first) return;
    race.enter(noise ? of_key(q) / divisor - logf(noise[i]) : of_key(q), q, static_cast<uint32_t>(i));
  });
  race.block_join<NT>(bins);
  return race.key ? Drawn{race.key, race.index} : Drawn{best, first};
}

// The winner, or where no score is a number the first item.
template <int NT>
__device__ __forceinline__ Drawn settle(Race &race, uint32_t best, uint32_t first, uint64_t *bins, uint64_t *tmp) {
  race.block_join<NT>(bins);
  if (race.key) return Drawn{race.key, race.index};
  return Drawn{best, ~static_cast<uint32_t>(block_max<NT>(static_cast<uint64_t>(~first), tmp))};
}

// The last item, in order of rank, above which the items at or above `lower`
// total less than `target` (counts, or masses), as a list has it; 0 if there
// is none.  Linear bins of log2 w (`per` to one, so that few lanes meet in one),
// then the items of the edge's bin, sorted.  False if those are too many.
template <bool kMassed, int NT, typename Items>
__device__ bool find_edge(const Items &items, Scale sc, float per_unit, uint64_t lower, uint64_t target, uint64_t *buf,
                          uint64_t *edge_list, int *listed, uint64_t *tmp, uint64_t &last) {
  uint32_t *bins = reinterpret_cast<uint32_t *>(buf);
  const auto bin_of = [&](uint32_t q) {
    return min(static_cast<int>((sc.top - of_key(q)) * sc.f * per_unit), kBins - 1);  // the conversion saturates
  };
  const auto counts = [&](int i, uint32_t q) {
    return q != 0 && (static_cast<uint64_t>(q) << 32 | ~static_cast<uint32_t>(i)) >= lower;
  };
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += NT) bins[i] = 0;
  if (threadIdx.x == 0) *listed = 0;
  __syncthreads();
  items.each([&](int i, uint32_t q) {
    if (counts(i, q)) atomicAdd(&bins[bin_of(q)], kMassed ? sc.mass(of_key(q)) : 1u);
  });
  __syncthreads();
  constexpr int per = kBins / NT;
  uint64_t mine = 0;
#pragma unroll
  for (int j = 0; j < per; ++j) mine += bins[threadIdx.x * per + j];
  uint64_t run = block_before<NT>(mine, tmp);
  int edge = -1;
  uint64_t edge_above = 0;
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const uint32_t c = bins[threadIdx.x * per + j];
    if (c != 0 && run < target) edge = threadIdx.x * per + j, edge_above = run;
    run += c;
  }
  const int bin = static_cast<int>(block_max<NT>(static_cast<uint64_t>(edge + 1), tmp)) - 1;
  if (bin < 0) {
    last = 0;
    return true;
  }
  if (edge == bin) tmp[16] = edge_above;
  __syncthreads();
  const uint64_t above = tmp[16];
  items.each([&](int i, uint32_t q) {
    if (counts(i, q) && bin_of(q) == bin) {
      const int at = atomicAdd(listed, 1);
      if (at < NT) edge_list[at] = static_cast<uint64_t>(q) << 32 | ~static_cast<uint32_t>(i);
    }
  });
  __syncthreads();
  const int n = *listed;
  if (n > NT) return false;
  int size = kWave;
  while (size < n) size <<= 1;
  const uint64_t c = block_sort<NT, uint64_t>(static_cast<int>(threadIdx.x) < n ? edge_list[threadIdx.x] : 0ull, size, buf);
  const bool real = static_cast<int>(threadIdx.x) < n;
  run = above + block_before<NT>(real ? (kMassed ? sc.mass(of_key(static_cast<uint32_t>(c >> 32))) : 1u) : 0u, tmp);
  // the lowest in rank of those below the target; complemented, so that it is the largest
  last = ~block_max<NT>(real && run < target ? ~c : 0ull, tmp);
  return true;
}

// The kept prefix and its race, over a list or a row, with find_edge.  all,
// as for select_prefix.  False if an edge lies among too many equal items.
template <int NT, typename Items>
__device__ bool select_edges(const Items &items, Scale sc, float per_unit, Filters flt, float divisor, const float *noise,
                             bool all, uint64_t *buf, uint64_t *edge_list, int *listed, uint64_t *tmp, Drawn &drawn) {
  uint64_t last = 0;
  if (flt.k > 0 && !find_edge<false, NT>(items, sc, per_unit, 0, static_cast<uint64_t>(flt.k), buf, edge_list, listed, tmp, last))
    return false;
  if (flt.p < 1.f) {
    uint64_t total = 0;
    items.each([&](int i, uint32_t q) {
      if (q != 0 && (static_cast<uint64_t>(q) << 32 | ~static_cast<uint32_t>(i)) >= last) total += sc.mass(of_key(q));
    });
    total = block_sum<NT>(total, tmp);
    if (flt.k == 0 && !all) total = static_cast<uint64_t>(kUnits);
    uint64_t edge;
    if (!find_edge<true, NT>(items, sc, per_unit, last, share_of(total, flt.p), buf, edge_list, listed, tmp, edge)) return false;
    if (edge != 0) last = edge;
  }
  const uint32_t best = key_of(sc.top);
  uint32_t first = 0xffffffffu;
  Race race;
  items.each([&](int i, uint32_t q) {
    if (q == best) first = min(first, static_cast<uint32_t>(i));
    if (q == 0 || (static_cast<uint64_t>(q) << 32 | ~static_cast<uint32_t>(i)) < last) return;
    const float y = of_key(q);
    if (sc.weight(y) >= flt.min) race.enter(noise ? y / divisor - logf(noise[i]) : y, q, static_cast<uint32_t>(i));
  });
  drawn = settle<NT>(race, best, first, buf, tmp);
  return true;
}

// The race over the items of a row that `kept(y)` says stay, and that have
// min-p's weight; `seen(i, y)` is called for every item.  first: the lowest index of the best score.
template <typename T, int NT, typename Kept, typename Seen>
__device__ void race_row(const RowItems<T, NT> &row, Scale sc, float least, float divisor, const float *noise, Race &race,
                         uint32_t &first, Kept stays, Seen seen) {
  using G = Granule<T>;
  row.each_granule([&](int at, const G &g) {
    uint32_t kept = 0;
#pragma unroll
    for (int j = 0; j < G::N; ++j) {
      const float y = g.at(j);
      if (y == sc.top) first = min(first, static_cast<uint32_t>(at + j));
      if (stays(y) && sc.weight(y) >= least) kept |= 1u << j;
      seen(at + j, y);
    }
    while (kept) {  // few of a granule's items are kept: as many turns as the lane with the most has
      const int i = at + __builtin_ctz(kept);
      kept &= kept - 1;
      const float x = clean(static_cast<float>(row.x[i]));
      race.enter(x / divisor - logf(noise[i]), item_key(x), i);
    }
  });
}

// Top-p alone, for rows whose prefix is long: masses by linear bins of
// log2 w (1/64 wide, so that few lanes meet in one; a histogram of float
// bits has its items in a few dozen); then the bins above the edge's race, while the items of the edge's
// bin go to a list, whose kept ones, once sorted, race too.  False if those are too many (equal scores).
template <typename T, int NT>
__device__ bool select_share(const RowItems<T, NT> &items, Scale sc, Filters flt, float divisor, const float *noise,
                             uint64_t *buf, uint64_t *list, int *listed, uint64_t *tmp, Drawn &drawn) {
  uint32_t *bins = reinterpret_cast<uint32_t *>(buf);
  const auto bin_of = [&](float y) {
    return min(static_cast<int>((sc.top - y) * sc.f * 64.f), kBins - 1);  // the conversion saturates
  };
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += NT) bins[i] = 0;
  if (threadIdx.x == 0) *listed = 0;
  __syncthreads();
  // All items below `far` together hold less than top-p leaves out: they can't
  // be at the edge, and are most of a long row.
  const float far = fminf(log2f(static_cast<float>(items.items) * sc.units / (kUnits * (1.f - flt.p))) + 0.01f, 1e9f);
  uint32_t total = 0;  // all masses together are 2^31, less or more their rounding
  items.each_score([&](int, float y) {
    const uint32_t m = sc.mass(y);  // 0 for -inf
    total += m;
    if ((sc.top - y) * sc.f < far) atomicAdd(&bins[bin_of(y)], m);
  });
  const uint64_t goal = share_of(block_sum<NT>(static_cast<uint64_t>(total), tmp), flt.p);
  __syncthreads();
  constexpr int per = kBins / NT;
  uint64_t mine = 0;
#pragma unroll
  for (int j = 0; j < per; ++j) mine += bins[threadIdx.x * per + j];
  uint64_t run = block_before<NT>(mine, tmp);
  int edge = -1;  // the last bin with any mass whose items have less than the goal above them
  uint64_t edge_above = 0;
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const uint32_t c = bins[threadIdx.x * per + j];
    if (c != 0 && run < goal) edge = threadIdx.x * per + j, edge_above = run;
    run += c;
  }
  const int bin = static_cast<int>(block_max<NT>(static_cast<uint64_t>(edge + 1), tmp)) - 1;
  if (edge == bin) tmp[16] = edge_above;
  __syncthreads();
  const uint64_t above = tmp[16];
  Race race;
  uint32_t first = 0xffffffffu;
  race_row(
      items, sc, flt.min, divisor, noise, race, first, [&](float y) { return bin_of(y) < bin && y > -__builtin_inff(); },
      [&](int i, float y) {
        if (bin_of(y) == bin && y > -__builtin_inff()) {
          const int at = atomicAdd(listed, 1);
          if (at < NT) list[at] = static_cast<uint64_t>(key_of(y)) << 32 | ~static_cast<uint32_t>(i);
        }
      });
  __syncthreads();
  const int n = *listed;
  if (n > NT) return false;
  int size = kWave;
  while (size < n) size <<= 1;
  const uint64_t c = block_sort<NT, uint64_t>(static_cast<int>(threadIdx.x) < n ? list[threadIdx.x] : 0ull, size, buf);
  const bool real = static_cast<int>(threadIdx.x) < n;
  mine = real ? sc.mass(of_key(static_cast<uint32_t>(c >> 32))) : 0;
  run = above + block_before<NT>(mine, tmp);
  if (real && run < goal) {
    const float y = of_key(static_cast<uint32_t>(c >> 32));
    const uint32_t i = ~static_cast<uint32_t>(c);
    if (sc.weight(y) >= flt.min) race.enter(y / divisor - logf(noise[i]), static_cast<uint32_t>(c >> 32), i);
  }
  drawn = settle<NT>(race, key_of(sc.top), first, buf, tmp);
  return true;
}

// kOne: an item per thread covers the row, and the sort takes it as it is.
// Longer rows are read again by each pass, which the caches serve (held in
// registers, granules spilled; held in LDS, a third to all of a row, every
// measured case took as long or longer).
template <typename T, int NT, bool kOne>
__global__ void __launch_bounds__(NT) sample_kernel(SampleArgs a) {
  using G = Granule<T>;
  __shared__ uint64_t bins[kBins / 2 > 2 * NT ? kBins / 2 : 2 * NT];  // a histogram, or a sort's buffers
  __shared__ uint64_t list[kOne ? 1 : kList];
  __shared__ uint64_t edge_list[kOne ? 1 : NT];
  __shared__ uint64_t tmp[17];
  __shared__ int listed;
  constexpr int kCap = sizeof(list) / 8;
  const int64_t r = a.first + blockIdx.x;
  const int tid = threadIdx.x, items = static_cast<int>(a.items);
  const T *x = static_cast<const T *>(a.scores) + r * a.stride;
  const float *noise = a.noise + r * a.noise_stride;
  const float t = a.temperature ? a.temperature[r] : 1.f;
  const bool greedy = !(t > 0.f);
  const float divisor = greedy ? 1.f : t;
  Filters flt{a.top_k ? a.top_k[r] : 0, a.top_p ? a.top_p[r] : 1.f, a.min_p ? a.min_p[r] : 0.f};
  if (flt.k < 0 || flt.k >= items) flt.k = 0;
  if (!(flt.p < 1.f)) flt.p = 1.f;
  if (greedy) flt = Filters{items > 1 ? 1 : 0, 1.f, 0.f};
  const bool open = !greedy && flt.k == 0 && flt.p == 1.f && !(flt.min > 0.f);  // every item may win
  // not 0, where -inf x 0 is no number: at an infinite temperature scores within 3.4e38 of the best weigh 1 (less 2^-21
  // at the most), -inf 0
  const float f = fminf(fmaxf(kLog2e / divisor, 1.401298464e-45f), kMost);

  // 1. maxima, and the sum of w against the thread's own maximum
  float mine = -__builtin_inff(), ref = -kMost, sum = 0.f;
  auto take = [&](const G &g) {
    float y[G::N], top = mine;
#pragma unroll
    for (int j = 0; j < G::N; ++j) {
      y[j] = g.at(j);
      top = fmaxf(top, y[j]);
    }
    mine = top;
    const float now = fmaxf(ref, top);
    sum *= __builtin_amdgcn_exp2f((ref - now) * f);
    ref = now;
#pragma unroll
    for (int j = 0; j < G::N; ++j) sum += __builtin_amdgcn_exp2f((y[j] - ref) * f);
  };
  const RowItems<T, NT> row{x, items};
  Race race;
  uint64_t own = 0;  // kOne: this thread's item, as a list has it
  if constexpr (kOne) {
    const float y = tid < items ? clean(static_cast<float>(x[tid])) : -__builtin_inff();
    mine = y;
    ref = fmaxf(ref, y);
    sum = __builtin_amdgcn_exp2f((y - ref) * f);
    if (item_key(y) != 0) own = static_cast<uint64_t>(key_of(y)) << 32 | ~static_cast<uint32_t>(tid);
    if (open && own != 0) race.enter(y / divisor - logf(noise[tid]), key_of(y), tid);
  } else if (open) {
    for (int first = tid * G::N; first < items; first += NT * G::N) {
      G g;
      float e[G::N];
      if (first <= items - G::N) {
        g.load(x, first, items);
        __builtin_memcpy(e, noise + first, sizeof(e));
      } else {
        g.load_end(x, first, items);
#pragma unroll
        for (int j = 0; j < G::N; ++j) e[j] = first + j < items ? noise[first + j] : 1.f;
      }
      take(g);
#pragma unroll
      for (int j = 0; j < G::N; ++j) {
        const float y = g.at(j);
        if (y > -__builtin_inff()) race.enter(y / divisor - logf(e[j]), key_of(y), first + j);
      }
    }
  } else {
    row.each_granule([&](int, const G &g) { take(g); });
  }
  const uint32_t best = static_cast<uint32_t>(block_max<NT>(static_cast<uint64_t>(item_key(mine)), tmp));
  if (best == 0) {
    if (tid == 0) {
      a.index[r] = -1;
      a.logprob[r] = -__builtin_inff();
    }
    return;
  }
  sum = block_sum<NT>(sum * __builtin_amdgcn_exp2f((ref - of_key(best)) * f), tmp);
  const Scale sc{of_key(best), f, kUnits / (flt.k > 0 ? fminf(sum, static_cast<float>(flt.k)) : sum)};

  Drawn drawn{best, 0};
  if (open) {
    race.block_join<NT>(bins);
    drawn = Drawn{race.key, race.index};
    if (race.key == 0) {  // no score is a number (the noise is not): the first item
      uint32_t first = own >> 32 == best ? static_cast<uint32_t>(tid) : 0xffffffffu;
      if constexpr (!kOne)
        for (int i = tid; i < items; i += NT)
          if (item_key(clean(static_cast<float>(x[i]))) == best) first = min(first, static_cast<uint32_t>(i));
      drawn = Drawn{best, ~static_cast<uint32_t>(block_max<NT>(static_cast<uint64_t>(~first), tmp))};
    }
  } else {
    // 2. the bound, and the list of the items that reach it
    uint32_t rank_bound = 1, min_bound = 1;
    bool by_rank = true, by_min = false;  // which bounds are worth a list
    if constexpr (!kOne) {
      const int owners = min(NT, items / G::N);
      const int rank = flt.k > 0 ? flt.k : owners / 2;
      if (rank <= owners && (flt.k > 0 || flt.p < 1.f)) {
        uint32_t *buf = reinterpret_cast<uint32_t *>(bins);
        uint32_t m = item_key(mine);
        int size = NT;
        if (flt.k > 0 && flt.k <= NT / 8 && owners == NT) {  // maxima of four threads will do: fewer to sort
          m = max(m, from_lane_xor<1>(m));
          m = max(m, from_lane_xor<2>(m));
          __syncthreads();
          if (tid % 4 == 0) buf[tid / 4] = m;
          __syncthreads();
          size = NT / 4 < kWave ? kWave : NT / 4;
          m = tid < NT / 4 ? buf[tid] : 0u;
        }
        m = block_sort<NT, uint32_t>(m, size, buf);
        __syncthreads();
        if (tid == rank - 1) tmp[16] = m;
        __syncthreads();
        rank_bound = max(static_cast<uint32_t>(tmp[16]), 1u);
        // without top-k the list has to reach top-p's share: its items weigh about 1.4 times their threads' maxima
        if (flt.k == 0) {
          const float some = block_sum<NT>(tid < rank && m != 0 ? sc.weight(of_key(m)) : 0.f, tmp);
          by_rank = 2.f * some >= flt.p * sum;
        }
      }
      // a little below min-p's own bound (its test follows per item); top-p's share of the first k needs all of those
      if (flt.min > 0.f && !(flt.k > 0 && flt.p < 1.f)) {
        min_bound = max(min(item_key(clean(sc.top + (log2f(flt.min) - 0.01f) / f)), best), 1u);
        // the list overflows (6,144 items) where nearly every thread's maximum reaches the bound
        const uint64_t reach = block_sum<NT>(static_cast<uint64_t>(item_key(mine) >= min_bound), tmp);
        by_min = static_cast<int>(reach) * 256 <= owners * 255;
      }
      if (flt.k == 0 && flt.p == 1.f) by_rank = false;
    }
    // with the rank's bound first; where that list doesn't hold the prefix, with min-p's own
    bool whole = false;
    for (int attempt = 0; attempt < 2 && !whole; ++attempt) {
      const uint32_t bound = attempt == 0 ? max(rank_bound, min_bound) : min_bound;
      if (attempt == 0 ? !by_rank : !by_min || (by_rank && min_bound >= rank_bound)) continue;
      __syncthreads();
      if (tid == 0) listed = 0;
      __syncthreads();
      const float floor = of_key(bound);
      if constexpr (!kOne)
        row.each_granule([&](int first, const G &g) {
          float y[G::N], top = -__builtin_inff();
#pragma unroll
          for (int j = 0; j < G::N; ++j) {
            y[j] = g.at(j);
            top = fmaxf(top, y[j]);
          }
          if (bound == 1 ? top > -__builtin_inff() : top >= floor) {
#pragma unroll
            for (int j = 0; j < G::N; ++j) {
              const uint32_t k = item_key(y[j]);
              if (k >= bound) {
                const int at = atomicAdd(&listed, 1);
                if (at < kCap) list[at] = static_cast<uint64_t>(k) << 32 | ~static_cast<uint32_t>(first + j);
              }
            }
          }
        });
      __syncthreads();
      const int n = kOne ? items : listed;
      whole = kOne || n <= kCap;  // the list holds every item that reaches the bound
      if (whole && n <= NT) {
        // 3. the sorted list
        int size = kWave;
        while (size < n) size <<= 1;
        const uint64_t c = block_sort<NT, uint64_t>(kOne ? own : tid < n ? list[tid] : 0ull, size, bins);
        const uint32_t key = static_cast<uint32_t>(c >> 32), at = ~static_cast<uint32_t>(c);
        const bool real = key != 0;
        const float y = real ? of_key(key) : 0.f, w = real ? sc.weight(y) : 0.f;
        float incl = w;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
          const float z = __shfl_up(incl, o);
          if (lane_id() >= o) incl += z;
        }
        float *waves = reinterpret_cast<float *>(tmp);
        __syncthreads();
        if (lane_id() == kWave - 1) waves[tid / kWave] = incl;
        __syncthreads();
        float before = incl - w, all = 0.f;
        for (int v = 0; v < NT / kWave; ++v) {
          if (v < tid / kWave) before += waves[v];
          all += waves[v];
        }
        float mass = sum;  // what top-p is a share of
        if (flt.k > 0 && flt.p < 1.f) {
          // the mass of the first k, or of all there are
          if (tid == min(flt.k, size) - 1) tmp[16] = __builtin_bit_cast(uint32_t, before + w);
          __syncthreads();
          mass = __builtin_bit_cast(float, static_cast<uint32_t>(tmp[16]));
        }
        // without top-k the list has to reach top-p's share, or min-p's bound
        whole = flt.k > 0 || bound == 1 || all >= flt.p * mass ||
                (min_bound > 1 && bound == min_bound);
        if (whole) {
          const bool keep = real && (tid == 0 || ((flt.k == 0 || tid < flt.k) &&
                                                  (flt.p == 1.f || before < flt.p * mass) && w >= flt.min));
          uint64_t run = 0;
          if (keep) {
            const float s = greedy ? y : y / divisor - logf(noise[at]);
            if (s == s) run = static_cast<uint64_t>(key_of(s)) << 32 | ~static_cast<uint32_t>(tid);
          }
          run = block_max<NT>(run, tmp);
          const int winner = run ? static_cast<int>(~static_cast<uint32_t>(run)) : 0;
          __syncthreads();
          if (tid == winner) tmp[16] = c;
          __syncthreads();
          drawn = Drawn{static_cast<uint32_t>(tmp[16] >> 32), ~static_cast<uint32_t>(tmp[16])};
        }
      } else if (!kOne && whole) {
        // a longer list: it has to hold the prefix, as above
        ListItems<NT> li{list, n};
        float all = 0.f;
        li.each([&](int, uint32_t q) { all += sc.weight(of_key(q)); });
        all = block_sum<NT>(all, tmp);
        whole = flt.k > 0 || bound == 1 || all >= flt.p * sum || (min_bound > 1 && bound == min_bound);
        // bins over what the list spans
        const float per_unit = fminf((kBins - 1) / fmaxf((sc.top - of_key(bound)) * sc.f, 1e-3f), 1e6f);
        if (whole && !select_edges<NT>(li, sc, bound == 1 ? 64.f : per_unit, flt, divisor, greedy ? nullptr : noise, bound == 1,
                                       bins, edge_list, &listed, tmp, drawn))
          drawn = select_prefix<NT>(li, sc, flt, divisor, greedy ? nullptr : noise, bound == 1, bins, tmp);
      }
    }
    if constexpr (!kOne)
      if (!whole) {
        if (flt.k == 0 && flt.p == 1.f) {
          uint32_t first = 0xffffffffu;
          race_row(row, sc, flt.min, divisor, noise, race, first, [](float y) { return y > -__builtin_inff(); }, [](int, float) {});
          drawn = settle<NT>(race, best, first, bins, tmp);
        } else if (flt.k > 0 ? !select_edges<NT>(row, sc, 64.f, flt, divisor, greedy ? nullptr : noise, true, bins, edge_list,
                                                 &listed, tmp, drawn)
                             : !select_share(row, sc, flt, divisor, noise, bins, list, &listed, tmp, drawn))
          drawn = select_prefix<NT>(row, sc, flt, divisor, greedy ? nullptr : noise, true, bins, tmp);
      }
  }
  if (tid == 0) {
    a.index[r] = drawn.index;
    a.logprob[r] = (of_key(drawn.key) - sc.top) / divisor - logf(sum);
  }
}

template <typename T, int NT, bool kOne>
hlr_status launch_rows(SampleArgs a, int64_t rows, hipStream_t stream) {
  for (; a.first < rows; a.first += most_blocks(NT)) {
    const int64_t here = rows - a.first < most_blocks(NT) ? rows - a.first : most_blocks(NT);
    sample_kernel<T, NT, kOne><<<static_cast<unsigned>(here), NT, 0, stream>>>(a);
    const hlr_status st = launch_status();
    if (st != HLR_OK) return st;
  }
  return HLR_OK;
}

// Threads by the row's length: one item per thread where the row is that
// short; 512 up to 8,192 items (64 rows of 8,192 fp16: top-k 50 12 us, 16 with 1,024; top-p
// 0.95 27 and 35), 1,024 beyond (128 rows of 16,384 fp32: top-k 900 29 us, 42 with 512; the
// others within 12%).
template <typename T>
hlr_status launch(const SampleArgs &a, int64_t rows, hipStream_t stream) {
  if (a.items <= 256) return launch_rows<T, 256, true>(a, rows, stream);
  if (a.items <= 512) return launch_rows<T, 512, true>(a, rows, stream);
  if (a.items <= 1024) return launch_rows<T, 1024, true>(a, rows, stream);
  if (a.items <= 8192) return launch_rows<T, 512, false>(a, rows, stream);
  return launch_rows<T, 1024, false>(a, rows, stream);
}

}  // namespace

extern "C" hlr_status sample_scores(const void *scores, int32_t type, int64_t rows, int64_t items, int64_t stride,
                                    const float *noise, int64_t noise_stride, const float *temperature,
                                    const int32_t *top_k, const float *top_p, const float *min_p, int64_t *out_index,
                                    float *out_logprob, hipStream_t stream) {
  if (rows < 0 || rows > kMaxN || items < 0 || items > HLR_SAMPLE_MAX_ITEMS || type < 0 || type > 2 || stride < 0 ||
      noise_stride < 0)
    return HLR_INVALID_ARG;
  if (rows == 0) return HLR_OK;
  if (!out_index || !out_logprob || (items > 0 && (!scores || !noise))) return HLR_INVALID_ARG;
  if (!aligned(scores, type == HLR_FP32 ? 4 : 2) || !aligned(noise, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(out_index, 8) || !aligned(out_logprob, 4))
    return HLR_MISALIGNED;
  const SampleArgs a{scores, stride, noise, noise_stride, temperature, top_k, top_p, min_p, items, out_index, out_logprob, 0};
  if (type == HLR_FP32) return launch<float>(a, rows, stream);
  if (type == HLR_BF16) return launch<bf16>(a, rows, stream);
  return launch<_Float16>(a, rows, stream);
}
