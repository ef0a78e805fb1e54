// A user's event history held in 8 bits: block tables and slot maps from
// request lengths, the quantising write and the read back.
//
// Layout (one pool of blocks for all requests): keys int8
// [blocks][heads][B][D], values int8 [blocks][heads][B/16][D][16], one fp32
// scale per block and head for each.  Values keep 16 tokens of one element
// together, so that the attention's second product reads its operand (for one
// d, consecutive tokens) as 16-byte loads straight into registers.
#include "hlr_common.hpp"
#include "hist_common.hpp"

#include <type_traits>

namespace {
using namespace hlr;

// ------------------------------------------------------------------ plan
// With c_r cached and n_r new tokens, request r's new blocks are columns
// ceil(c_r/B) .. ceil((c_r+n_r)/B)-1 of its table row and come from the free
// list in request order, so everything follows from two exclusive prefix sums
// over the requests (tokens and new blocks).  One launch: every block scans
// the lengths for itself into LDS (at most 4,096 groups of 2^shift requests)
// and then maps its own tile of tokens by a binary search; a scan is a few
// thousand integer additions from L2, less than a second launch costs.  A new
// block begins with a new token, so the thread of that token writes the
// table entry.  Latency bound: 3.8 us for 64 requests, 13 us for 4,096 with a
// map of 250,000 places (lengths, scan, search and table one after another).
constexpr int kPlanThreads = 512;
constexpr int kPlanTile = 2048;
constexpr int kPlanGroups = 4096;

__device__ __forceinline__ int sat32(int64_t x) { return x > 0x7fffffff ? 0x7fffffff : static_cast<int>(x); }

__device__ __forceinline__ int length_after(int cached, int fresh) {
  return sat32(static_cast<int64_t>(max(cached, 0)) + max(fresh, 0));
}

// The new lengths alone, in the place of cached or fresh: every block of
// plan_kernel reads those, so they are written by a launch after it.
__global__ void __launch_bounds__(256) lengths_kernel(const int *cached, const int *fresh, int R, int *lengths) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r < R) lengths[r] = length_after(cached[r], fresh[r]);
}

// kGroups: groups of 2^group_shift requests, whose lengths are read again
// where a token falls into one; otherwise every request has its own entry and its length is kept in LDS.
template <bool kGroups>
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const int *__restrict__ cached, const int *__restrict__ fresh, int R, int *__restrict__ table,
                int64_t cols, const int *__restrict__ free_blocks, int64_t num_free, int log_b, int group_shift,
                int64_t max_tokens, int64_t *__restrict__ slots, int *__restrict__ cu, int *__restrict__ lengths,
                int64_t *__restrict__ counts) {
  __shared__ int tok_first[kPlanGroups];  // tokens before the group, saturated (first: a request's new tokens)
  __shared__ int blk_first[kPlanGroups];  // new blocks before the group, saturated
  __shared__ int held_in[kGroups ? 1 : kPlanGroups];
  __shared__ int64_t wave_tok[kPlanThreads / kWave], wave_blk[kPlanThreads / kWave], wave_lost[kPlanThreads / kWave];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int shift = kGroups ? group_shift : 0;
  const int groups = (R + (1 << shift) - 1) >> shift;
  const int per = (groups + kPlanThreads - 1) / kPlanThreads;  // groups of a thread
  const int g0 = min(tid * per, groups), g1 = min(g0 + per, groups);
  const int r0 = min(g0 << shift, R), r1 = min(g1 << shift, R);
  const int64_t bmask = (int64_t(1) << log_b) - 1;
  if constexpr (!kGroups) {
    for (int r = tid; r < R; r += kPlanThreads) {
      held_in[r] = max(cached[r], 0);
      tok_first[r] = max(fresh[r], 0);
    }
    __syncthreads();
  }
  const auto cached_of = [&](int r) -> int64_t { return kGroups ? max(cached[r], 0) : held_in[r]; };

  int64_t tok = 0, blk = 0;
  for (int r = r0; r < r1; ++r) {
    const int64_t c = cached_of(r), n = kGroups ? max(fresh[r], 0) : tok_first[r];
    tok += n;
    blk += ((c + n + bmask) >> log_b) - ((c + bmask) >> log_b);
  }
  int64_t tok_in = tok, blk_in = blk;  // inclusive over the wave
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t a = __shfl_up(tok_in, o), b = __shfl_up(blk_in, o);
    if (lane >= o) tok_in += a, blk_in += b;
  }
  if (lane == kWave - 1) wave_tok[wave] = tok_in, wave_blk[wave] = blk_in;
  __syncthreads();
  int64_t tok_at = tok_in - tok, blk_at = blk_in - blk, total = 0, total_blk = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / kWave; ++w) {
    if (w < wave) tok_at += wave_tok[w], blk_at += wave_blk[w];
    total += wave_tok[w], total_blk += wave_blk[w];
  }
  const bool writes = blockIdx.x == gridDim.x - 1;  // the last block has the fewest tokens
  int64_t lost = 0;
  for (int g = g0; g < g1; ++g) {
    const int own = tok_first[g];
    tok_first[g] = sat32(tok_at);
    blk_first[g] = sat32(blk_at);
    for (int r = g << shift; r < min((g + 1) << shift, R); ++r) {
      const int64_t c = cached_of(r), n = kGroups ? max(fresh[r], 0) : own;
      const int64_t col = (c + bmask) >> log_b, need = ((c + n + bmask) >> log_b) - col;
      if (writes) {
        cu[r] = sat32(tok_at);
        if (lengths) lengths[r] = sat32(c + n);
        // tokens that find no block: the open block's, then those of new blocks
        const int64_t open = min(n, (col << log_b) - c);
        if (open > 0 && !(c >> log_b < cols && table[r * cols + (c >> log_b)] >= 0)) lost += open;
        const int64_t have = min(min(need, max(num_free - blk_at, int64_t(0))), max(cols - col, int64_t(0)));
        lost += max(n - open - (have << log_b), int64_t(0));
      }
      tok_at += n;
      blk_at += need;
    }
  }
  if (writes) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) lost += __shfl_xor(lost, o);
    if (lane == 0) wave_lost[wave] = lost;
  }
  __syncthreads();
  if (writes && tid == 0) {
    for (int w = 1; w < kPlanThreads / kWave; ++w) lost += wave_lost[w];
    cu[R] = sat32(total);
    counts[0] = min(total_blk, num_free);
    counts[1] = lost;
  }
  // two tokens at a time, so that their searches and loads run side by side
  constexpr int kSide = 2;
  for (int i = tid; i < kPlanTile; i += kSide * kPlanThreads) {
    int64_t slot[kSide];
#pragma unroll
    for (int v = 0; v < kSide; ++v) {
      const int64_t t = static_cast<int64_t>(blockIdx.x) * kPlanTile + i + v * kPlanThreads;
      slot[v] = -1;
      if (t >= max_tokens || t >= total) continue;
      int lo = 0, hi = groups - 1;  // the last group that begins at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tok_first[mid] <= t)
          lo = mid;
        else
          hi = mid - 1;
      }
      int r = lo << shift;
      int64_t first = tok_first[lo], fb = blk_first[lo], c = cached_of(r);
      if constexpr (kGroups) {
        int64_t n = max(fresh[r], 0);
        while (t >= first + n) {  // the last group that begins at or before t holds t
          fb += ((c + n + bmask) >> log_b) - ((c + bmask) >> log_b);
          first += n;
          ++r;
          c = max(cached[r], 0);
          n = max(fresh[r], 0);
        }
      }
      const int64_t p = c + (t - first), col = p >> log_b, held = (c + bmask) >> log_b;
      if (col < cols) {
        int64_t b;
        if (col < held) {
          b = table[r * cols + col];
        } else {
          const int64_t at = fb + (col - held);
          b = at < num_free ? free_blocks[at] : -1;
          if ((p & bmask) == 0) table[r * cols + col] = static_cast<int>(b);
        }
        if (b >= 0) slot[v] = (b << log_b) + (p & bmask);
      }
    }
#pragma unroll
    for (int v = 0; v < kSide; ++v) {
      const int64_t t = static_cast<int64_t>(blockIdx.x) * kPlanTile + i + v * kPlanThreads;
      if (t < max_tokens) slots[t] = slot[v];
    }
  }
}

// ------------------------------------------------- runs of consecutive slots
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kSpan = 64;  // tokens that a block looks through

// Bit i: token t0 + i follows token t0 + i - 1 in the next slot of the same
// group of 2^log_g slots (so a run goes on); a bit that is not set begins a
// run, or is a token without a slot in the pool.  `slot` receives this lane's
// token's slot (-1 outside).
__device__ __forceinline__ uint64_t follows(const int64_t *slots, int64_t t0, int64_t tokens, int64_t num_slots, int log_g,
                                            int64_t &slot) {
  const int64_t t = t0 + lane_id();
  slot = t < tokens ? slots[t] : -1;
  const int64_t prev = t > 0 && t <= tokens ? slots[t - 1] : -1;
  if (slot >= num_slots) slot = -1;
  return ballot(slot > 0 && prev == slot - 1 && (slot & ((1 << log_g) - 1)) != 0);
}

// ---------------------------------------------------------------- append
// Per block and head, over the run of new values x that falls into it:
//   s' = max(s, fl(amax|x| * fl(1/127)))   (s counts only if the block holds tokens)
//   held codes, where s' > s: rne(fl(q * fl(s * fl(1/s'))))
//   new codes: clamp(rne(fl(x * fl(1/s'))), -127, 127)
// One block of threads owns a run, so nothing is atomic and the result does
// not depend on the order of the blocks.  A run is the longest sequence of
// tokens in consecutive slots of one cache block; each thread block looks for
// the runs that begin in its span of tokens, by ballots.
//
// A run's values are read with 16-byte loads for the keys (a thread has 16
// elements of a token, and stores 16 codes) and, for the values, as two
// elements of each of 16 tokens: a wave then reads whole rows, and a thread's
// 16 codes of one element are one store.  A thread holds its first units between
// the maximum and the codes; the rest of a large block (over 128 elements x 64
// tokens) is read again, from the caches.  73,700 tokens x 8 heads x 128
// bf16: 130 us, 3.5 TB/s of keys and values in and codes out, bound by loads in
// flight (115 registers, four waves per SIMD); one token for each of 256 requests: 9 us.
// The low byte of the result is the code of x (clamped, rounded to nearest
// even by adding 1.5 * 2^23, whose steps are whole); NaN gives 0.
__device__ __forceinline__ uint32_t code(float x, float inv) {
  const float y = __builtin_amdgcn_fmed3f((x == x ? x : 0.f) * inv, -127.f, 127.f);
  return __builtin_bit_cast(uint32_t, y + 12582912.f);
}
// Likewise for a held code (a byte at bit `sh` of w) times a ratio below 1.
__device__ __forceinline__ uint32_t scaled(uint32_t w, int sh, float ratio) {
  const float y = static_cast<float>(static_cast<int8_t>(w >> sh)) * ratio;
  return __builtin_bit_cast(uint32_t, y + 12582912.f);
}
__device__ __forceinline__ uint32_t four_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(b, a, 0x0c0c0400u) | __builtin_amdgcn_perm(d, c, 0x0c0c0400u) << 16;
}
__device__ __forceinline__ u4 scaled16(u4 c, float ratio) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = four_bytes(scaled(c[i], 0, ratio), scaled(c[i], 8, ratio), scaled(c[i], 16, ratio), scaled(c[i], 24, ratio));
  return c;
}

// Element i of packed elements.
template <typename T>
__device__ __forceinline__ float element(const uint32_t *w, int i) {
  if constexpr (sizeof(T) == 4)
    return __builtin_bit_cast(float, w[i]);
  else if constexpr (std::is_same<T, bf16>::value)
    return __builtin_bit_cast(float, i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  else
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16))));
}

struct AppendArgs {
  const void *x[2];          // keys, values
  int64_t tok_stride[2], head_stride[2];
  int8_t *codes[2];
  float *scale[2];
  const int64_t *slots;
  int64_t tokens, num_slots;
  int heads, log_b, span;
  int64_t first;  // span of this launch's first blocks
};

// 16 elements of one token.
template <typename T>
struct Sixteen {
  uint32_t w[4 * sizeof(T)];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) {
      const u4 y = reinterpret_cast<const u4 *>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = y[j];
    }
  }
  __device__ __forceinline__ float at(int j) const { return element<T>(w, j); }
  __device__ __forceinline__ float top() const {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(at(j)));
    return m;
  }
};

// Two elements of the 16 tokens of a chunk; zeros where the run has none.
template <typename T>
struct Chunk {
  static constexpr int W = sizeof(T) / 2;
  uint32_t w[16 * W];
  // p: the elements in the run's first token; at: the chunk's first place less the run's.
  __device__ __forceinline__ void load(const T *p, int64_t stride, int at, int len) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const bool in = at + j >= 0 && at + j < len;
      const uint32_t *y = reinterpret_cast<const uint32_t *>(p + (at + j) * stride);
#pragma unroll
      for (int i = 0; i < W; ++i) w[j * W + i] = in ? y[i] : 0u;
    }
  }
  __device__ __forceinline__ float at(int j, int which) const { return element<T>(w + j * W, which); }
  __device__ __forceinline__ float top() const {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = fmaxf(m, fmaxf(fabsf(at(j, 0)), fabsf(at(j, 1))));
    return m;
  }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(NT) append_kernel(AppendArgs a) {
  // keys and values of all heads next to each other in the grid, as they are in a token's row
  const int which = blockIdx.x / a.heads % 2, head = blockIdx.x % a.heads, tid = threadIdx.x, lane = lane_id();
  const int B = 1 << a.log_b;
  const T *x = static_cast<const T *>(a.x[which]) + head * a.head_stride[which];
  const int64_t stride = a.tok_stride[which];
  __shared__ float top[2][NT / kWave];
  int turn = 0;
  const int64_t t0 = (a.first + blockIdx.x / (2 * a.heads)) * a.span;
  int64_t my_slot;
  const uint64_t goes_on = follows(a.slots, t0, a.tokens, a.num_slots, a.log_b, my_slot);
  uint64_t starts = ~goes_on & ballot(my_slot >= 0);
  if (a.span < kSpan) starts &= (1ull << a.span) - 1;
  while (starts) {
    const int at0 = __builtin_ctzll(starts);
    starts &= starts - 1;
    const int64_t t = t0 + at0, slot = readlane_i64(my_slot, at0);
    // the run ends at the next token that doesn't follow, in this window of 64 or a later one
    const uint64_t rest = at0 == 63 ? 0 : ~goes_on >> (at0 + 1);
    int len = rest ? __builtin_ctzll(rest) + 1 : 64 - at0;
    if (!rest || at0 + len >= 64)
      while (true) {
        int64_t s;
        const uint64_t more = follows(a.slots, t + len, a.tokens, a.num_slots, a.log_b, s);
        if (~more) {
          len += __builtin_ctzll(~more);
          break;
        }
        len += 64;
      }
    const int first = static_cast<int>(slot & (B - 1));
    const int64_t bh = (slot >> a.log_b) * a.heads + head;
    const T *xr = x + t * stride;
    float *sp = a.scale[which] + bh;
    const float old = first > 0 ? *sp : 0.f;
    int8_t *q = a.codes[which] + ((bh << a.log_b) * D);

    // the largest magnitude of the run (NaN drops out)
    float m = 0.f;
    constexpr int kParts = D / 16, kPairs = D / 2;
    constexpr int kHeld = sizeof(T) == 4 ? 1 : 2, kHeldV = 1;  // units held, 16 registers each or 32
    const int c0 = first / 16, units = which == 0 ? len * kParts : ((first + len + 15) / 16 - c0) * kPairs;
    Sixteen<T> ky[kHeld];
    Chunk<T> vy[kHeldV];
    if (which == 0) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        const int u = tid + h * NT;
        if (u < units) ky[h].load(xr + (u / kParts) * stride + (u % kParts) * 16), m = fmaxf(m, ky[h].top());
      }
      for (int u = tid + kHeld * NT; u < units; u += NT) {
        Sixteen<T> y;
        y.load(xr + (u / kParts) * stride + (u % kParts) * 16);
        m = fmaxf(m, y.top());
      }
    } else {
#pragma unroll
      for (int h = 0; h < kHeldV; ++h) {
        const int u = tid + h * NT, at = (c0 + u / kPairs) * 16 - first;  // the chunk's place in the run
        if (u < units) vy[h].load(xr + u % kPairs * 2, stride, at, len), m = fmaxf(m, vy[h].top());
      }
      for (int u = tid + kHeldV * NT; u < units; u += NT) {
        Chunk<T> y;
        y.load(xr + u % kPairs * 2, stride, (c0 + u / kPairs) * 16 - first, len);
        m = fmaxf(m, y.top());
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if constexpr (NT > kWave) {
      if (lane == 0) top[turn][tid / kWave] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NT / kWave; ++w) m = fmaxf(m, top[turn][w]);
      turn ^= 1;
    }
    float now = fminf(m, 3.402823466e38f) * (1.f / 127.f);
    if (now < 1.17549435e-38f) now = 0.f;  // below the normal range: the values are stored as zeros
    now = fmaxf(now, old);
    const float inv = now > 0.f ? 1.f / now : 0.f;
    const bool grown = first > 0 && now > old;
    const float ratio = old * inv;
    if (tid == 0) *sp = now;

    if (which == 0) {
      if (grown)
        for (int u = tid; u < first * kParts; u += NT) {
          u4 *w = reinterpret_cast<u4 *>(q) + u;
          *w = scaled16(*w, ratio);
        }
      const auto put = [&](int u, const Sixteen<T> &y) {
        u4 c;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c[i] = four_bytes(code(y.at(4 * i), inv), code(y.at(4 * i + 1), inv), code(y.at(4 * i + 2), inv),
                            code(y.at(4 * i + 3), inv));
        reinterpret_cast<u4 *>(q)[first * kParts + u] = c;
      };
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (tid + h * NT < units) put(tid + h * NT, ky[h]);
      for (int u = tid + kHeld * NT; u < units; u += NT) {
        Sixteen<T> y;
        y.load(xr + (u / kParts) * stride + (u % kParts) * 16);
        put(u, y);
      }
    } else {
      if (grown)  // whole chunks of held tokens; the one that the run begins in follows with the run
        for (int u = tid; u < c0 * D; u += NT) {
          u4 *w = reinterpret_cast<u4 *>(q) + u;
          *w = scaled16(*w, ratio);
        }
      const auto put = [&](int u, const Chunk<T> &v) {
        const int c = c0 + u / kPairs, d = u % kPairs * 2;
        const int lo = first - c * 16, hi = lo + len;  // the run's places in the chunk
        u4 *w = reinterpret_cast<u4 *>(q + (c * D + d) * 16);
        uint32_t n0[16], n1[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) n0[j] = code(v.at(j, 0), inv), n1[j] = code(v.at(j, 1), inv);
        u4 y0, y1;
        if (lo > 0 || hi < 16) {  // places outside the run keep their codes, or held ones are rounded again
          y0 = w[0];
          y1 = w[1];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int sh = j % 4 * 8;
            if (j >= lo && j < hi) continue;
            n0[j] = grown && j < lo ? scaled(y0[j / 4], sh, ratio) : y0[j / 4] >> sh;
            n1[j] = grown && j < lo ? scaled(y1[j / 4], sh, ratio) : y1[j / 4] >> sh;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y0[i] = four_bytes(n0[4 * i], n0[4 * i + 1], n0[4 * i + 2], n0[4 * i + 3]);
          y1[i] = four_bytes(n1[4 * i], n1[4 * i + 1], n1[4 * i + 2], n1[4 * i + 3]);
        }
        w[0] = y0;
        w[1] = y1;
      };
#pragma unroll
      for (int h = 0; h < kHeldV; ++h)
        if (tid + h * NT < units) put(tid + h * NT, vy[h]);
      for (int u = tid + kHeldV * NT; u < units; u += NT) {
        Chunk<T> y;
        y.load(xr + u % kPairs * 2, stride, (c0 + u / kPairs) * 16 - first, len);
        put(u, y);
      }
    }
  }
}

// ------------------------------------------------------------------ read
// Keys: 16 codes of a token per thread.  Values: a wave takes a run of tokens
// in one chunk of 16 slots, two elements per lane, so the chunk is read once
// with 16-byte loads and whole rows are written.  73,700 tokens x 8 heads x
// 128 to bf16: 90 to 110 us, 4.1 to 5 TB/s.
struct ReadArgs {
  const int8_t *codes[2];
  const float *scale[2];
  void *out[2];
  const int64_t *slots;
  int64_t tokens, num_slots;
  int heads, log_b;
  int64_t first;  // span of this launch's first blocks
};

template <typename T>
struct alignas(2 * sizeof(T)) Pair {
  T a[2];
};

template <typename T, int D>
__global__ void __launch_bounds__(256) read_kernel(ReadArgs a) {
  const int which = blockIdx.x / a.heads % 2, head = blockIdx.x % a.heads, tid = threadIdx.x;
  const int lane = lane_id(), wave = tid / kWave;
  T *out = static_cast<T *>(a.out[which]) + static_cast<int64_t>(head) * D;
  const int64_t row = static_cast<int64_t>(a.heads) * D, t0 = (a.first + blockIdx.x / (2 * a.heads)) * kSpan;
  const int here = static_cast<int>(min(static_cast<int64_t>(kSpan), a.tokens - t0));
  const int in_b = (1 << a.log_b) - 1;
  if (which == 0) {
    constexpr int kParts = D / 16;
#pragma unroll 2
    for (int u = tid; u < here * kParts; u += 256) {
      const int64_t t = t0 + u / kParts, slot = a.slots[t];
      u4 c = {0, 0, 0, 0};
      float s = 0.f;
      if (slot >= 0 && slot < a.num_slots) {
        const int64_t bh = (slot >> a.log_b) * a.heads + head;
        c = reinterpret_cast<const u4 *>(a.codes[0] + (((bh << a.log_b) + (slot & in_b)) * D))[u % kParts];
        s = a.scale[0][bh];
      }
      T y[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] = static_cast<T>(static_cast<float>(static_cast<int8_t>(c[j / 4] >> (j % 4 * 8))) * s);
      u4 raw[sizeof(T)];
      __builtin_memcpy(raw, y, sizeof(raw));
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) reinterpret_cast<u4 *>(out + t * row + (u % kParts) * 16)[i] = raw[i];
    }
    return;
  }
  constexpr int kLanes = D >= 128 ? 64 : D / 2;  // lanes of a run
  int64_t my_slot;
  const uint64_t goes_on = follows(a.slots, t0, a.tokens, a.num_slots, 4, my_slot);
  uint64_t starts = ~goes_on | 1;  // the span's first token begins a run here whatever came before it
  if (here < kSpan) starts &= (1ull << here) - 1;
  const uint64_t ends = starts >> 1;
  constexpr int kSide = kWave / kLanes;  // runs that a wave takes at a time
  int skip = wave * kSide + lane / kLanes;  // every (4 * kSide)-th run is this lane group's
  while (starts) {
    for (; skip > 0 && starts; --skip) starts &= starts - 1;
    if (!starts) break;
    const int at = __builtin_ctzll(starts);
    const uint64_t rest = ends >> at;
    const int len = rest ? min(__builtin_ctzll(rest) + 1, here - at) : here - at;
    const int64_t slot = a.slots[t0 + at];
    const bool real = slot >= 0 && slot < a.num_slots;
    const int64_t bh = real ? (slot >> a.log_b) * a.heads + head : 0;
    const float s = real ? a.scale[1][bh] : 0.f;
    const int place = real ? static_cast<int>(slot & 15) : 0;  // a token without a slot is a run of its own
#pragma unroll
    for (int part = 0; part < (D + 127) / 128; ++part) {
      const int d = part * 128 + lane % kLanes * 2;
      u4 y0 = {0, 0, 0, 0}, y1 = {0, 0, 0, 0};
      if (real) {
        const u4 *w = reinterpret_cast<const u4 *>(
            a.codes[1] + (((bh << (a.log_b - 4)) + ((slot & in_b) >> 4)) * D + d) * 16);
        y0 = w[0];
        y1 = w[1];
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (j < place || j >= place + len) continue;
        const int64_t t = t0 + at + j - place;
        Pair<T> v;
        v.a[0] = static_cast<T>(static_cast<float>(static_cast<int8_t>(y0[j / 4] >> (j % 4 * 8))) * s);
        v.a[1] = static_cast<T>(static_cast<float>(static_cast<int8_t>(y1[j / 4] >> (j % 4 * 8))) * s);
        *reinterpret_cast<Pair<T> *>(out + t * row + d) = v;
      }
    }
    skip = 4 * kSide;
  }
}

// Blocks of NT threads for keys and values, head by head, of each span of tokens.
template <int NT, typename A, typename Launch>
hlr_status launch_spans(A a, int64_t span, Launch launch) {
  const int64_t spans = grid_for(a.tokens, static_cast<int>(span)), most = most_blocks(NT) / (2 * a.heads);
  for (; a.first < spans; a.first += most) {
    const int64_t here = spans - a.first < most ? spans - a.first : most;
    launch(static_cast<unsigned>(here * 2 * a.heads), a);
    const hlr_status st = launch_status();
    if (st != HLR_OK) return st;
  }
  return HLR_OK;
}
template <typename T, int D>
hlr_status launch_append(const AppendArgs &a, hipStream_t stream) {
  // few tokens: a wave per token and head, since most runs are single tokens then; else a block per span
  if (a.span == 1)
    return launch_spans<64>(a, 1, [&](unsigned grid, const AppendArgs &b) { append_kernel<T, D, 64><<<grid, 64, 0, stream>>>(b); });
  return launch_spans<256>(a, a.span,
                           [&](unsigned grid, const AppendArgs &b) { append_kernel<T, D, 256><<<grid, 256, 0, stream>>>(b); });
}
template <typename T, int D>
hlr_status launch_read(const ReadArgs &a, hipStream_t stream) {
  return launch_spans<256>(a, kSpan, [&](unsigned grid, const ReadArgs &b) { read_kernel<T, D><<<grid, 256, 0, stream>>>(b); });
}
template <typename T>
hlr_status launch_append_dim(const AppendArgs &a, int64_t dim, hipStream_t stream) {
  switch (dim) {
    case 32: return launch_append<T, 32>(a, stream);
    case 64: return launch_append<T, 64>(a, stream);
    case 128: return launch_append<T, 128>(a, stream);
    default: return launch_append<T, 256>(a, stream);
  }
}
template <typename T>
hlr_status launch_read_dim(const ReadArgs &a, int64_t dim, hipStream_t stream) {
  switch (dim) {
    case 32: return launch_read<T, 32>(a, stream);
    case 64: return launch_read<T, 64>(a, stream);
    case 128: return launch_read<T, 128>(a, stream);
    default: return launch_read<T, 256>(a, stream);
  }
}

int log2_block(int64_t b) { return b == 16 ? 4 : b == 32 ? 5 : b == 64 ? 6 : b == 128 ? 7 : b == 256 ? 8 : -1; }

hlr_status check_cache(const void *kc, const void *vc, const void *ks, const void *vs, int64_t num_blocks, int64_t heads,
                       int64_t block, int64_t dim) {
  if (num_blocks < 0 || num_blocks > kMaxN || heads <= 0 || heads > 65535 || log2_block(block) < 0) return HLR_INVALID_ARG;
  if (dim != 32 && dim != 64 && dim != 128 && dim != 256) return HLR_UNSUPPORTED_DIM;
  if (num_blocks > 0 && (!kc || !vc || !ks || !vs)) return HLR_INVALID_ARG;
  if (!aligned(kc, 16) || !aligned(vc, 16) || !aligned(ks, 4) || !aligned(vs, 4)) return HLR_MISALIGNED;
  return HLR_OK;
}

}  // namespace

extern "C" hlr_status hist_plan(const int32_t *cached, const int32_t *fresh, int64_t requests, int32_t *block_table,
                                int64_t table_cols, const int32_t *free_blocks, int64_t num_free, int64_t block,
                                int64_t max_tokens, int64_t *out_slots, int32_t *out_cu, int32_t *out_lengths,
                                int64_t *out_counts, hipStream_t stream) {
  const int log_b = log2_block(block);
  if (requests < 0 || requests > HLR_HIST_MAX_REQUESTS || table_cols < 0 || table_cols > kMaxN || num_free < 0 ||
      num_free > kMaxN || max_tokens < 0 || max_tokens > kMaxN || log_b < 0)
    return HLR_INVALID_ARG;
  if (!out_cu || !out_counts || (requests > 0 && (!cached || !fresh || !out_lengths)) ||
      (requests > 0 && table_cols > 0 && !block_table) || (num_free > 0 && !free_blocks) ||
      (max_tokens > 0 && !out_slots))
    return HLR_INVALID_ARG;
  if (!aligned(cached, 4) || !aligned(fresh, 4) || !aligned(block_table, 4) || !aligned(free_blocks, 4) ||
      !aligned(out_slots, 8) || !aligned(out_cu, 4) || !aligned(out_lengths, 4) || !aligned(out_counts, 8))
    return HLR_MISALIGNED;
  // every block reads the inputs while others write: no output may lie in one, except the lengths in place
  const bool in_place = requests > 0 && (out_lengths == cached || out_lengths == fresh);
  const struct {
    const void *at;
    int64_t bytes;
    bool out;
  } spans[] = {{cached, 4 * requests, false},          {fresh, 4 * requests, false}, {free_blocks, 4 * num_free, false},
               {block_table, 4 * requests * table_cols, true}, {out_slots, 8 * max_tokens, true},
               {out_cu, 4 * (requests + 1), true},     {out_counts, 16, true},
               {out_lengths, in_place ? 0 : 4 * requests, true}};
  for (const auto &x : spans)
    for (const auto &y : spans)
      if (&x != &y && x.out && x.bytes > 0 && y.bytes > 0) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(x.at), b = reinterpret_cast<uintptr_t>(y.at);
        if (a < b + y.bytes && b < a + x.bytes) return HLR_INVALID_ARG;
      }
  int shift = 0;
  while ((requests + (int64_t(1) << shift) - 1) >> shift > kPlanGroups) ++shift;
  const int grid = grid_for(max_tokens, kPlanTile), R = static_cast<int>(requests);
  int *lengths = in_place ? nullptr : out_lengths;
  if (shift == 0)
    plan_kernel<false><<<grid, kPlanThreads, 0, stream>>>(cached, fresh, R, block_table, table_cols, free_blocks, num_free,
                                                          log_b, shift, max_tokens, out_slots, out_cu, lengths, out_counts);
  else
    plan_kernel<true><<<grid, kPlanThreads, 0, stream>>>(cached, fresh, R, block_table, table_cols, free_blocks, num_free,
                                                         log_b, shift, max_tokens, out_slots, out_cu, lengths, out_counts);
  const hlr_status st = launch_status();
  if (st != HLR_OK || !in_place) return st;
  lengths_kernel<<<grid_for(requests, 256), 256, 0, stream>>>(cached, fresh, R, out_lengths);
  return launch_status();
}

extern "C" hlr_status hist_append(int8_t *k_codes, int8_t *v_codes, float *k_scale, float *v_scale, int64_t num_blocks,
                                  int64_t heads, int64_t block, int64_t dim, const void *k, const void *v,
                                  int32_t type, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                  int64_t v_head_stride, const int64_t *slots, int64_t tokens, hipStream_t stream) {
  const hlr_status st = check_cache(k_codes, v_codes, k_scale, v_scale, num_blocks, heads, block, dim);
  if (st != HLR_OK) return st;
  if (tokens < 0 || tokens > kMaxN || type < 0 || type > 2) return HLR_INVALID_ARG;
  if (tokens == 0) return HLR_OK;
  if (!k || !v || !slots) return HLR_INVALID_ARG;
  const int64_t unit = type == HLR_FP32 ? 4 : 8;  // elements of 16 bytes
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || k_token_stride % unit || k_head_stride % unit ||
      v_token_stride % unit || v_head_stride % unit)
    return HLR_MISALIGNED;
  AppendArgs a{{k, v}, {k_token_stride, v_token_stride}, {k_head_stride, v_head_stride}, {k_codes, v_codes},
               {k_scale, v_scale}, slots, tokens, num_blocks * block, static_cast<int>(heads), log2_block(block), 1, 0};
  while (a.span < kSpan && tokens * heads * 2 / a.span > 8192) a.span *= 2;
  if (type == HLR_FP32) return launch_append_dim<float>(a, dim, stream);
  if (type == HLR_BF16) return launch_append_dim<bf16>(a, dim, stream);
  return launch_append_dim<_Float16>(a, dim, stream);
}

extern "C" hlr_status hist_read(const int8_t *k_codes, const int8_t *v_codes, const float *k_scale,
                                const float *v_scale, int64_t num_blocks, int64_t heads, int64_t block, int64_t dim,
                                const int64_t *slots, int64_t tokens, void *out_k, void *out_v, int32_t type,
                                hipStream_t stream) {
  const hlr_status st = check_cache(k_codes, v_codes, k_scale, v_scale, num_blocks, heads, block, dim);
  if (st != HLR_OK) return st;
  if (tokens < 0 || tokens > kMaxN || type < 0 || type > 2) return HLR_INVALID_ARG;
  if (tokens == 0) return HLR_OK;
  if (!slots || !out_k || !out_v) return HLR_INVALID_ARG;
  if (!aligned(slots, 8) || !aligned(out_k, 16) || !aligned(out_v, 16)) return HLR_MISALIGNED;
  const ReadArgs a{{k_codes, v_codes}, {k_scale, v_scale}, {out_k, out_v}, slots, tokens, num_blocks * block,
                   static_cast<int>(heads), log2_block(block), 0};
  if (type == HLR_FP32) return launch_read_dim<float>(a, dim, stream);
  if (type == HLR_BF16) return launch_read_dim<bf16>(a, dim, stream);
  return launch_read_dim<_Float16>(a, dim, stream);
}
