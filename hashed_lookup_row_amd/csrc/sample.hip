// Sampling one item per row of scores with temperature, top-k, top-p and
// min-p, from given random numbers.
//
// z = x / temperature; items rank by (z descending, index ascending); the
// filters keep a prefix of that order:
//   top-k  the first k
//   top-p  item i while the mass of the items before it is below top_p times
//          the mass of the first k    (mass: w = exp(z - max z))
//   min-p  w >= min_p
// and always the first item.  Of the kept items the one with the largest
// z - log(noise) is drawn (noise ~ Exp(1): an exponential race, so item i wins
// with probability w_i over the kept mass).
//
// A prefix is a threshold key and a number of items kept of those equal to it
// (in index order), so nothing is sorted: a row is read once into registers
// (rows that do not fit are read again for each pass), and a radix selection over the
// order-preserving integer of z finds the key by counts (top-k) or by masses
// (top-p).  Masses are summed as whole numbers of 2^-36, so the result does
// not depend on the order of the additions.  Only the kept items' noise is
// read.  One block per row.
#include "hlr_common.hpp"
#include "hist_common.hpp"

namespace {
using namespace hlr;

constexpr float kMass = 68719476736.f;  // 2^36
constexpr int kBins = 2048;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __builtin_bit_cast(uint32_t, z + 0.f);  // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __builtin_bit_cast(float, (k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

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
};

template <typename T, int NT, int E>
struct Row {
  static constexpr int kWavesN = NT / kWave;
  const T *x;
  int items;
  float temperature;
  bool divide;
  uint32_t held[E > 0 ? E : 1];

  // key of item i: 0 for items that can't be drawn (NaN, -inf)
  __device__ __forceinline__ uint32_t make(int i) const {
    float z = static_cast<float>(x[i]);
    if (divide) z = z / temperature;
    return z > -__builtin_inff() ? key_of(fminf(z, 3.402823466e38f)) : 0u;
  }
  __device__ __forceinline__ void load() {
    if constexpr (E > 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = e * NT + threadIdx.x;
        held[e] = i < items ? make(i) : 0u;
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if constexpr (E > 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) f(e * NT + threadIdx.x, held[e]);
    } else {
      for (int i = threadIdx.x; i < items; i += NT) f(i, make(i));
    }
  }
};

template <int NT>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *tmp) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o)));
  if (lane_id() == 0) tmp[threadIdx.x / kWave] = v;
  __syncthreads();
  v = tmp[0];
#pragma unroll
  for (int w = 1; w < NT / kWave; ++w) v = max(v, tmp[w]);
  __syncthreads();
  return v;
}

template <int NT>
__device__ __forceinline__ float block_sum(float v, uint32_t *tmp) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if (lane_id() == 0) tmp[threadIdx.x / kWave] = __builtin_bit_cast(uint32_t, v);
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w) v += __builtin_bit_cast(float, tmp[w]);
  __syncthreads();
  return v;
}

template <int NT>
__device__ __forceinline__ uint64_t block_sum64(uint64_t v, uint64_t *tmp) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if (lane_id() == 0) tmp[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w) v += tmp[w];
  __syncthreads();
  return v;
}

__device__ __forceinline__ float weight(uint32_t key, float top) {
  return __builtin_amdgcn_exp2f((of_key(key) - top) * kLog2e);
}
__device__ __forceinline__ uint64_t mass_of(float w) { return static_cast<uint64_t>(__builtin_rintf(w * kMass)); }

// Finds, among the items with key >= floor, the key t at which the total
// of the items above it is still below `target` while that of the items at or
// above it reaches it (or the lowest key there is); `above` receives the total above t.
// Totals are counts (kMassed false) or masses.
template <bool kMassed, typename R, int NT>
__device__ uint32_t select_key(const R &row, uint32_t floor, float top, uint64_t target, uint64_t *bins, uint64_t *tmp,
                               uint64_t &above) {
  uint32_t prefix = 0, mask = 0;
  above = 0;
  const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = shifts[pass];
    const uint32_t field = (1u << widths[pass]) - 1u;
    for (int i = threadIdx.x; i < kBins; i += NT) bins[i] = 0;
    __syncthreads();
    row.each([&](int, uint32_t k) {
      if (k != 0 && k >= floor && (k & mask) == prefix)
        atomicAdd(reinterpret_cast<unsigned long long *>(&bins[(k >> shift) & field]),
                  static_cast<unsigned long long>(kMassed ? mass_of(weight(k, top)) : 1));
    });
    __syncthreads();
    // the lowest bin (bins descend in rank) whose total above is below the target and that is not empty
    constexpr int per = kBins / NT > 0 ? kBins / NT : 1;
    uint64_t mine = 0;
    const int b0 = kBins - 1 - threadIdx.x * per;
#pragma unroll
    for (int j = 0; j < per; ++j)
      if (b0 - j >= 0) mine += bins[b0 - j];
    uint64_t incl = mine;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const uint64_t y = __shfl_up(incl, o);
      if (lane_id() >= o) incl += y;
    }
    if (lane_id() == kWave - 1) tmp[threadIdx.x / kWave] = incl;
    if (threadIdx.x == 0) tmp[16] = ~0ull;
    __syncthreads();
    uint64_t before = above + incl - mine;
    for (int w = 0; w < static_cast<int>(threadIdx.x) / kWave; ++w) before += tmp[w];
    // candidates: non-empty bins with total above < target; the lowest wins, i.e. the largest descending position
    int best = -1;
    uint64_t best_above = 0, run = before;
#pragma unroll
    for (int j = 0; j < per; ++j)
      if (b0 - j >= 0) {
        const uint64_t c = bins[b0 - j];
        if (c != 0 && run < target) best = kBins - 1 - (b0 - j), best_above = run;
        run += c;
      }
    __syncthreads();
    uint32_t *t32 = reinterpret_cast<uint32_t *>(tmp);
    const uint32_t win = block_max<NT>(static_cast<uint32_t>(best + 1), t32);
    if (best >= 0 && static_cast<uint32_t>(best + 1) == win) tmp[16] = best_above;
    __syncthreads();
    if (win == 0) return 0;  // nothing there
    above = tmp[16];
    const uint32_t bin = kBins - win;
    prefix |= bin << shift;
    mask |= field << shift;
    __syncthreads();
  }
  return prefix;
}

template <typename T, int NT, int E>
__global__ void __launch_bounds__(NT) sample_kernel(SampleArgs a) {
  using R = Row<T, NT, E>;
  __shared__ uint64_t bins[kBins];
  __shared__ uint64_t tmp64[17];
  __shared__ uint32_t cut;
  __shared__ uint64_t race_key[NT / kWave];
  __shared__ uint32_t race_z[NT / kWave];
  uint32_t *tmp = reinterpret_cast<uint32_t *>(tmp64);
  const int64_t r = blockIdx.x;
  const int items = static_cast<int>(a.items);
  R row;
  row.x = static_cast<const T *>(a.scores) + r * a.stride;
  row.items = items;
  row.temperature = a.temperature ? a.temperature[r] : 1.f;
  const bool race = row.temperature > 0.f;
  row.divide = race && row.temperature != 1.f;
  row.load();

  uint32_t best = 0;
  row.each([&](int, uint32_t k) { best = max(best, k); });
  best = block_max<NT>(best, tmp);
  if (best == 0) {
    if (threadIdx.x == 0) {
      a.index[r] = -1;
      a.logprob[r] = -__builtin_inff();
    }
    return;
  }
  const float top = of_key(best);
  float sum = 0.f;
  uint32_t first = 0xffffffffu;  // the first item: the lowest index of the best key
  row.each([&](int i, uint32_t k) {
    if (k != 0) sum += weight(k, top);
    if (k == best) first = min(first, static_cast<uint32_t>(i));
  });
  sum = block_sum<NT>(sum, tmp);
  first = ~block_max<NT>(~first, tmp);

  uint32_t drawn = first, drawn_key = best;
  if (race) {
    // the kept prefix: keys above `edge`, and of those equal to it the first `ties` by index
    uint32_t edge = 1;
    uint64_t ties = 0xffffffffu;
    const int k = a.top_k ? a.top_k[r] : 0;
    if (k > 0 && k < items) {
      uint64_t above;
      const uint32_t t = select_key<false, R, NT>(row, 1, top, static_cast<uint64_t>(k), bins, tmp64, above);
      edge = t;
      ties = static_cast<uint64_t>(k) - above;
    }
    const float p = a.top_p ? a.top_p[r] : 1.f;
    if (p < 1.f) {
      // the mass of the first k: all above the edge, and `ties` of the items at it (or all, if fewer)
      uint64_t over = 0, at_edge = 0;
      row.each([&](int, uint32_t q) {
        if (q > edge) over += mass_of(weight(q, top));
        if (q == edge) ++at_edge;
      });
      over = block_sum64<NT>(over, tmp64);
      at_edge = block_sum64<NT>(at_edge, tmp64);
      if (at_edge > 0) over += min(at_edge, ties) * mass_of(weight(edge, top));
      const double target = static_cast<double>(p) * static_cast<double>(over);
      uint64_t goal = target > 1.0 ? static_cast<uint64_t>(target) : 1;  // the first item stays
      uint64_t above;
      const uint32_t t = select_key<true, R, NT>(row, edge, top, goal, bins, tmp64, above);
      if (t != 0) {
        const uint64_t w = mass_of(weight(t, top));
        const uint64_t n = w > 0 ? (goal - above + w - 1) / w : 0xffffffffull;
        if (t > edge)
          ties = n;
        else
          ties = n < ties ? n : ties;
        edge = t;
      }
    }
    // items equal to the edge: how many there are, and where the kept ones end
    uint32_t equal = 0;
    row.each([&](int, uint32_t q) { equal += q == edge; });
    equal = static_cast<uint32_t>(block_sum64<NT>(equal, tmp64));
    uint32_t last = 0xffffffffu;
    if (equal > ties) {
      if (threadIdx.x == 0) cut = 0xffffffffu;
      __syncthreads();
      uint32_t seen = 0;
      for (int base = 0; base < items && seen < ties; base += NT) {
        const int i = base + threadIdx.x;
        const bool is = i < items && row.make(i) == edge;
        const uint64_t m = ballot(is);
        if (lane_id() == 0) tmp[threadIdx.x / kWave] = __popcll(m);
        __syncthreads();
        uint32_t before = seen, all = 0;
        for (int w = 0; w < NT / kWave; ++w) {
          if (w < static_cast<int>(threadIdx.x) / kWave) before += tmp[w];
          all += tmp[w];
        }
        before += __popcll(m & lanemask_lt());
        if (is && before + 1 == ties) cut = static_cast<uint32_t>(i);
        seen += all;
        __syncthreads();
      }
      last = cut;
    }
    const float least = a.min_p ? a.min_p[r] : 0.f;
    const float *noise = a.noise + r * a.noise_stride;
    // the race: by z - log(noise), then by rank
    float s_best = -__builtin_inff();
    uint32_t i_best = first, k_best = best;
    bool any = false;
    row.each([&](int i, uint32_t q) {
      if (q < edge || q == 0) return;
      if (q == edge && static_cast<uint32_t>(i) > last) return;
      if (q != best && !(weight(q, top) >= least)) return;
      if (q == best && static_cast<uint32_t>(i) != first && !(1.f >= least)) return;
      const float s = of_key(q) - logf(noise[i]);
      const bool better = !any || s > s_best || (s == s_best && (q > k_best || (q == k_best && static_cast<uint32_t>(i) < i_best)));
      if (better && s == s) {
        s_best = s;
        i_best = static_cast<uint32_t>(i);
        k_best = q;
        any = true;
      }
    });
    uint64_t packed = any ? (static_cast<uint64_t>(key_of(s_best)) << 32 | ~i_best) : 0ull;
    // over the wave and the block, in order of (score, key, index)
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t y = __shfl_xor(packed, o);
      const uint32_t yk = static_cast<uint32_t>(__shfl_xor(static_cast<int>(k_best), o));
      const uint32_t ps = packed >> 32, ys = y >> 32;
      if (ys > ps || (ys == ps && (yk > k_best || (yk == k_best && y > packed)))) packed = y, k_best = yk;
    }
    if (lane_id() == 0) race_key[threadIdx.x / kWave] = packed, race_z[threadIdx.x / kWave] = k_best;
    __syncthreads();
    packed = race_key[0];
    k_best = race_z[0];
    for (int w = 1; w < NT / kWave; ++w) {
      const uint64_t y = race_key[w];
      const uint32_t yk = race_z[w];
      const uint32_t ps = packed >> 32, ys = y >> 32;
      if (ys > ps || (ys == ps && (yk > k_best || (yk == k_best && y > packed)))) packed = y, k_best = yk;
    }
    if (packed != 0) {
      drawn = ~static_cast<uint32_t>(packed);
      drawn_key = k_best;
    }
  }
  if (threadIdx.x == 0) {
    a.index[r] = drawn;
    a.logprob[r] = (of_key(drawn_key) - top) - logf(sum);
  }
}

template <typename T>
void launch(const SampleArgs &a, int64_t rows, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(rows);
  if (a.items <= 256 * 8)
    sample_kernel<T, 256, 8><<<grid, 256, 0, stream>>>(a);
  else if (a.items <= 1024 * 32)
    sample_kernel<T, 1024, 32><<<grid, 1024, 0, stream>>>(a);
  else
    sample_kernel<T, 1024, 0><<<grid, 1024, 0, stream>>>(a);
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
  const SampleArgs a{scores, stride, noise, noise_stride, temperature, top_k, top_p, min_p, items, out_index, out_logprob};
  if (type == HLR_FP32)
    launch<float>(a, rows, stream);
  else if (type == HLR_BF16)
    launch<bf16>(a, rows, stream);
  else
    launch<_Float16>(a, rows, stream);
  return launch_status();
}
