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
// table entry.
constexpr int kPlanThreads = 512;
constexpr int kPlanTile = 2048;
constexpr int kPlanGroups = 4096;

__device__ __forceinline__ int sat32(int64_t x) { return x > 0x7fffffff ? 0x7fffffff : static_cast<int>(x); }

__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const int *__restrict__ cached, const int *__restrict__ fresh, int R, int *__restrict__ table,
                int64_t cols, const int *__restrict__ free_blocks, int64_t num_free, int log_b, int group_shift,
                int64_t max_tokens, int64_t *__restrict__ slots, int *__restrict__ cu, int *__restrict__ lengths,
                int64_t *__restrict__ counts) {
  __shared__ int tok_first[kPlanGroups];  // tokens before the group, saturated
  __shared__ int blk_first[kPlanGroups];  // new blocks before the group, saturated
  __shared__ int64_t wave_tok[kPlanThreads / kWave], wave_blk[kPlanThreads / kWave], wave_lost[kPlanThreads / kWave];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int groups = (R + (1 << group_shift) - 1) >> group_shift;
  const int per = (groups + kPlanThreads - 1) / kPlanThreads;  // groups of a thread
  const int g0 = tid * per, g1 = min(g0 + per, groups);
  const int r0 = min(g0 << group_shift, R), r1 = min(g1 << group_shift, R);
  const int64_t bmask = (int64_t(1) << log_b) - 1;

  int64_t tok = 0, blk = 0;
  for (int r = r0; r < r1; ++r) {
    const int64_t c = max(cached[r], 0), n = max(fresh[r], 0);
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
  const bool writes = blockIdx.x == 0;
  int64_t lost = 0;
  for (int g = g0; g < g1; ++g) {
    tok_first[g] = sat32(tok_at);
    blk_first[g] = sat32(blk_at);
    for (int r = g << group_shift; r < min((g + 1) << group_shift, R); ++r) {
      const int64_t c = max(cached[r], 0), n = max(fresh[r], 0);
      const int64_t col = (c + bmask) >> log_b, need = ((c + n + bmask) >> log_b) - col;
      if (writes) {
        cu[r] = sat32(tok_at);
        lengths[r] = sat32(c + n);
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
  for (int i = tid; i < kPlanTile; i += kPlanThreads) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kPlanTile + i;
    if (t >= max_tokens) return;
    int64_t slot = -1;
    if (t < total) {
      int lo = 0, hi = groups - 1;  // the last group that begins at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tok_first[mid] <= t)
          lo = mid;
        else
          hi = mid - 1;
      }
      int r = lo << group_shift;
      int64_t first = tok_first[lo], fb = blk_first[lo];
      int64_t c = max(cached[r], 0), n = max(fresh[r], 0);
      while (t >= first + n) {  // within the group (the last group begins at or before t, so it holds t)
        fb += ((c + n + bmask) >> log_b) - ((c + bmask) >> log_b);
        first += n;
        ++r;
        c = max(cached[r], 0);
        n = max(fresh[r], 0);
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
        if (b >= 0) slot = (b << log_b) + (p & bmask);
      }
    }
    slots[t] = slot;
  }
}

// ---------------------------------------------------------------- append
// Per block and head, over the run of new values x that falls into it:
//   s' = max(s, fl(amax|x| * fl(1/127)))   (s counts only if the block holds tokens)
//   held codes, where s' > s: rne(fl(q * fl(s * fl(1/s'))))
//   new codes: clamp(rne(fl(x * fl(1/s'))), -127, 127)
// One block of threads owns a run, so nothing is atomic and the result does
// not depend on the order of the blocks.  A run is the longest sequence of
// tokens in consecutive slots of one block; each thread block looks for the
// runs that begin in its tile of tokens.
constexpr int kAppendThreads = 256;

template <typename T>
__device__ __forceinline__ float clean(T x) {
  const float v = static_cast<float>(x);
  if (v != v) return 0.f;
  return fminf(fmaxf(v, -3.402823466e38f), 3.402823466e38f);
}

__device__ __forceinline__ int code(float x, float inv) {
  return static_cast<int>(fminf(fmaxf(__builtin_rintf(x * inv), -127.f), 127.f));
}

struct AppendArgs {
  const void *x[2];          // keys, values
  int64_t tok_stride[2], head_stride[2];
  int8_t *codes[2];
  float *scale[2];
  const int64_t *slots;
  int64_t tokens, num_slots;
  int heads, dim, log_b, tile;
};

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a) {
  const int which = blockIdx.z, head = blockIdx.y, tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int B = 1 << a.log_b, D = a.dim;
  const T *x = static_cast<const T *>(a.x[which]) + head * a.head_stride[which];
  const int64_t stride = a.tok_stride[which];
  __shared__ float top[kAppendThreads / kWave];
  __shared__ int run_end;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile;
  for (int64_t t = t0; t < min(t0 + a.tile, a.tokens); ++t) {
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.num_slots) continue;
    const int first = static_cast<int>(slot & (B - 1));
    if (t > 0 && first != 0 && a.slots[t - 1] == slot - 1) continue;  // not the start of a run
    // length of the run
    __syncthreads();
    if (tid == 0) run_end = B - first;
    __syncthreads();
    const int most = static_cast<int>(min(static_cast<int64_t>(B - first), a.tokens - t));
    for (int i = tid; i < B - first; i += kAppendThreads)
      if (i >= most || a.slots[t + i] != slot + i) atomicMin(&run_end, i);
    __syncthreads();
    const int len = run_end;
    const int64_t block = slot >> a.log_b;
    const T *xr = x + t * stride;
    // the largest magnitude of the run
    float m = 0.f;
    for (int i = tid * 4; i < len * D; i += kAppendThreads * 4) {
      const T *p = xr + (i / D) * stride + (i % D);
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(clean(p[j])));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (lane == 0) top[wave] = m;
    float *sp = a.scale[which] + block * a.heads + head;
    const float old = first > 0 ? *sp : 0.f;
    __syncthreads();
    m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    float now = m * (1.f / 127.f);
    if (now < 1.17549435e-38f) now = 0.f;  // below the normal range: the values are stored as zeros
    now = fmaxf(now, old);
    const float inv = now > 0.f ? 1.f / now : 0.f;
    const bool grown = first > 0 && now > old;
    const float ratio = old * inv;
    if (tid == 0) *sp = now;
    int8_t *q = a.codes[which] + (block * a.heads + head) * (static_cast<int64_t>(B) * D);
    if (which == 0) {
      if (grown)
        for (int i = tid; i < first * D; i += kAppendThreads) q[i] = static_cast<int8_t>(__builtin_rintf(q[i] * ratio));
      for (int i = tid; i < len * D; i += kAppendThreads)
        q[first * D + i] = static_cast<int8_t>(code(clean(xr[(i / D) * stride + (i % D)]), inv));
    } else {
      // (16-token chunk, element) units: chunk bytes [D][16]
      const int c0 = grown ? 0 : first / 16, c1 = (first + len + 15) / 16;
      for (int u = tid; u < (c1 - c0) * D; u += kAppendThreads) {
        const int c = c0 + u / D, d = u % D;
        int8_t *w = q + (static_cast<int64_t>(c) * D + d) * 16;
        for (int j = 0; j < 16; ++j) {
          const int at = c * 16 + j;
          if (at < first) {
            if (grown) w[j] = static_cast<int8_t>(__builtin_rintf(w[j] * ratio));
          } else if (at < first + len) {
            w[j] = static_cast<int8_t>(code(clean(xr[(at - first) * stride + d]), inv));
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ read
struct ReadArgs {
  const int8_t *codes[2];
  const float *scale[2];
  void *out[2];
  const int64_t *slots;
  int64_t tokens, num_slots;
  int heads, dim, log_b;
};

template <typename T>
__global__ void __launch_bounds__(256) read_kernel(ReadArgs a) {
  const int which = blockIdx.z, D = a.dim;
  T *out = static_cast<T *>(a.out[which]);
  const int64_t n = a.tokens * a.heads * D, step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) {
    const int d = static_cast<int>(i % D);
    const int64_t th = i / D;
    const int h = static_cast<int>(th % a.heads);
    const int64_t slot = a.slots[th / a.heads];
    float v = 0.f;
    if (slot >= 0 && slot < a.num_slots) {
      const int64_t block = slot >> a.log_b;
      const int at = static_cast<int>(slot & ((1 << a.log_b) - 1));
      const int64_t bh = block * a.heads + h;
      const int8_t *q = a.codes[which] + ((bh << a.log_b) * D);
      const int8_t c = which == 0 ? q[at * D + d] : q[((at >> 4) * D + d) * 16 + (at & 15)];
      v = c * a.scale[which][bh];
    }
    out[i] = static_cast<T>(v);
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
  int shift = 0;
  while ((requests + (int64_t(1) << shift) - 1) >> shift > kPlanGroups) ++shift;
  plan_kernel<<<grid_for(max_tokens, kPlanTile), kPlanThreads, 0, stream>>>(
      cached, fresh, static_cast<int>(requests), block_table, table_cols, free_blocks, num_free, log_b, shift,
      max_tokens, out_slots, out_cu, out_lengths, out_counts);
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
               {k_scale, v_scale}, slots, tokens, num_blocks * block, static_cast<int>(heads), static_cast<int>(dim),
               log2_block(block), 1};
  while (a.tile < block && tokens * heads * 2 / a.tile > 8192) a.tile *= 2;
  const dim3 grid(grid_for(tokens, a.tile), static_cast<unsigned>(heads), 2);
  if (type == HLR_FP32)
    append_kernel<float><<<grid, kAppendThreads, 0, stream>>>(a);
  else if (type == HLR_BF16)
    append_kernel<bf16><<<grid, kAppendThreads, 0, stream>>>(a);
  else
    append_kernel<_Float16><<<grid, kAppendThreads, 0, stream>>>(a);
  return launch_status();
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
  ReadArgs a{{k_codes, v_codes}, {k_scale, v_scale}, {out_k, out_v}, slots, tokens, num_blocks * block,
             static_cast<int>(heads), static_cast<int>(dim), log2_block(block)};
  const int64_t want = (tokens * heads * dim + 255) / 256;
  const dim3 grid(static_cast<unsigned>(want < 16384 ? want : 16384), 1, 2);
  if (type == HLR_FP32)
    read_kernel<float><<<grid, 256, 0, stream>>>(a);
  else if (type == HLR_BF16)
    read_kernel<bf16><<<grid, 256, 0, stream>>>(a);
  else
    read_kernel<_Float16><<<grid, 256, 0, stream>>>(a);
  return launch_status();
}
