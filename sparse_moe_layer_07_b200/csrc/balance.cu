// The router's auxiliary losses: balance loss over the experts' shares of each
// sequence, z-loss, the per-sequence counts, and the gradient to the logits.
//
// With live tokens (unmasked, inside a sequence), n_s of them in sequence s and
// N in all, p_t = softmax(l_t), lse_t = log sum_e exp(l_te):
//   counts[s, e] = assignments of s's live tokens to e,  f_se = counts[s, e] / (2 n_s)
//   balance = E / N  sum_t sum_e f_{s(t) e} p_te          z = 1 / N  sum_t lse_t^2
//   d(a balance + b z) / d l_te = p_te (a E / N (f_se - sum_j f_sj p_tj) + 2 b / N lse_t)
// (f holds routing decisions and has no gradient).  The balance loss is a sum
// over tokens once the counts are known, so there are two passes: (1) counts
// from the choices and the mask alone, (2) one read of the logits that gives
// both losses and the gradient.  Every input is read once but the mask.
//
// Counts of sequences that cross token chunks: the pairs (chunk c, sequence s)
// that meet form a staircase, each step of which raises c or s, so c + s names
// a slot of its own; pass 1 writes the pair's counts there and pass 2 sums a
// sequence's slots.  Integers, so no order matters; the float sums run in a
// fixed order (thread, warp, chunk), so results do not depend on scheduling.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kE = 8;
constexpr int kChunk = 1024;   // tokens of a chunk
constexpr int kWindow = 1024;  // sequences whose counts are held at once (a chunk meets more only if most are empty)
constexpr int kSlot = 16;      // int32 of a slot: 8 counts, live tokens, padding to 64 bytes

struct BalanceArgs {
  const float* logits;         // [T, E]
  const int32_t* idx;          // [T, 2]
  const uint8_t* mask;         // [T] or NULL
  const int32_t* seq;          // [n_seq + 1] or NULL: one sequence of T tokens
  int64_t T;
  int32_t n_seq;
  int32_t n_chunks;            // ceil(T / kChunk), at least 1
  float a, b;                  // coefficients of the balance loss and the z-loss
  int32_t* counts;             // [n_seq, E]
  float* loss;                 // [3]: a balance + b z, balance, z
  float* dlogits;              // [T, E] or NULL
  int32_t* slots;              // [n_chunks + n_seq][kSlot]
  int32_t* chunk_live;         // [n_chunks]
  float2* chunk_sum;           // [n_chunks]: sum of sum_e f p, sum of lse^2
  int32_t* ticket;             // blocks of pass 2 that are done
  int* err;
};

__device__ __forceinline__ int bound_of(const BalanceArgs& a, int s) {
  const int64_t v = a.seq ? (int64_t)__ldg(a.seq + s) : (s == 0 ? 0 : a.T);
  return (int)(v < 0 ? 0 : (v > a.T ? a.T : v));
}

// Number of sequences in [lo, hi) that end at or before token t, plus lo: the
// sequence of t when t lies in one (empty sequences are passed over).
__device__ __forceinline__ int seq_of(const BalanceArgs& a, int t, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (bound_of(a, mid + 1) <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

template <int NT>
struct Shared {
  int hist[kWindow][kE + 1];  // pass 1: counts and live tokens; pass 2: f (as float bits) in [0, E)
  int first, last;            // sequences that tokens of the chunk can belong to
  int red[NT / 16][kSlot];
  float2 fred[NT / 32];
  int ired[NT / 32];
  int done;
};

// Sequence range [first, last] of chunk c; last < first when the chunk has no token in a sequence.
template <int NT>
__device__ __forceinline__ void chunk_range(const BalanceArgs& a, int c, Shared<NT>& sh) {
  if (threadIdx.x == 0 || threadIdx.x == 32) {
    const int begin = bound_of(a, 0), end = bound_of(a, a.n_seq);
    int64_t t0 = (int64_t)c * kChunk, t1 = t0 + kChunk;
    if (t1 > a.T) t1 = a.T;
    if (t0 < begin) t0 = begin;
    if (t1 > end) t1 = end;
    if (threadIdx.x == 0)
      sh.first = t0 < t1 ? seq_of(a, (int)t0, 0, a.n_seq) : 0;
    else
      sh.last = t0 < t1 ? seq_of(a, (int)t1 - 1, 0, a.n_seq) : -1;
  }
  __syncthreads();
}

// Sequence of token t of the chunk, or -1 for a token that does not count.
template <int NT>
__device__ __forceinline__ int live_seq(const BalanceArgs& a, int64_t t, const Shared<NT>& sh) {
  if (t >= a.T || sh.last < sh.first) return -1;
  if (t < bound_of(a, 0) || t >= bound_of(a, a.n_seq)) return -1;
  if (a.mask && !__ldg(a.mask + t)) return -1;
  const int s = seq_of(a, (int)t, sh.first, sh.last);
  return s < a.n_seq ? s : -1;
}

// Pass 1 over chunk c: counts of every sequence that meets the chunk, into its slot.
template <int NT>
__device__ __forceinline__ void count_chunk(const BalanceArgs& a, int c, Shared<NT>& sh) {
  constexpr int kTok = kChunk / NT;
  chunk_range(a, c, sh);
  const int first = sh.first, last = sh.last;
  int seq[kTok], e0[kTok], e1[kTok], live = 0;
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const int64_t t = (int64_t)c * kChunk + j * NT + threadIdx.x;
    seq[j] = live_seq(a, t, sh);
    e0[j] = e1[j] = -1;
    if (seq[j] >= 0) {
      const int2 p = __ldg(reinterpret_cast<const int2*>(a.idx) + t);
      e0[j] = p.x;
      e1[j] = p.y;
      if ((unsigned)p.x >= kE || (unsigned)p.y >= kE) flag_error(a.err, MOE_DEVERR_EXPERT_INDEX);
      ++live;
    }
  }
  for (int w0 = first; w0 <= last; w0 += kWindow) {
    const int n = min(last - w0 + 1, kWindow);
    for (int i = threadIdx.x; i < n * (kE + 1); i += NT) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    if (n == 1) {
      // one sequence: ballots instead of atomics on the same few words
#pragma unroll
      for (int e = 0; e <= kE; ++e) {
        int cnt = 0;
#pragma unroll
        for (int j = 0; j < kTok; ++j)
          cnt += e < kE ? __popc(__ballot_sync(~0u, seq[j] == w0 && e0[j] == e)) +
                              __popc(__ballot_sync(~0u, seq[j] == w0 && e1[j] == e))
                        : __popc(__ballot_sync(~0u, seq[j] == w0));
        if ((threadIdx.x & 31) == 0 && cnt) atomicAdd(&sh.hist[0][e], cnt);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        const int s = seq[j] - w0;
        if (seq[j] >= 0 && s >= 0 && s < n) {
          if ((unsigned)e0[j] < kE) atomicAdd(&sh.hist[s][e0[j]], 1);
          if ((unsigned)e1[j] < kE) atomicAdd(&sh.hist[s][e1[j]], 1);
          atomicAdd(&sh.hist[s][kE], 1);
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * (kE + 1); i += NT) {
      const int s = i / (kE + 1), q = i - s * (kE + 1);
      a.slots[((int64_t)c + w0 + s) * kSlot + q] = sh.hist[s][q];
    }
    __syncthreads();
  }
  const int warp_live = __reduce_add_sync(~0u, live);
  if ((threadIdx.x & 31) == 0) sh.ired[threadIdx.x >> 5] = warp_live;
  __syncthreads();
  if (threadIdx.x == 0) {
    int sum = 0;
    for (int w = 0; w < NT / 32; ++w) sum += sh.ired[w];
    a.chunk_live[c] = sum;
  }
}

// Chunk that writes the counts of sequence s: the one that holds its first token (empty ones: the place it would have).
__device__ __forceinline__ int owner_of(const BalanceArgs& a, int s) {
  const int c = bound_of(a, s) / kChunk;
  return c < a.n_chunks ? c : a.n_chunks - 1;
}

// Value q (counts, live tokens) of sequence s, summed over its slots from `at` on in steps.
__device__ __forceinline__ int sum_slots(const BalanceArgs& a, int s, int q, int at, int step) {
  const int lo = bound_of(a, s), hi = bound_of(a, s + 1);
  if (lo >= hi) return 0;
  int v = 0;
  const int c1 = (hi - 1) / kChunk;
#pragma unroll 4
  for (int c = lo / kChunk + at; c <= c1; c += step) v += __ldcg(a.slots + ((int64_t)c + s) * kSlot + q);
  return v;
}

// Pass 2 over chunk c: f of its sequences, then the tokens' losses and gradients.
template <int NT>
__device__ __forceinline__ void gradient_chunk(const BalanceArgs& a, int c, float inv_n, Shared<NT>& sh) {
  constexpr int kTok = kChunk / NT;
  chunk_range(a, c, sh);
  const int first = sh.first, last = sh.last;
  float sum_f = 0.f, sum_z = 0.f;
  float l[kTok][kE];
  int seq[kTok];
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const int64_t t = (int64_t)c * kChunk + j * NT + threadIdx.x;
    seq[j] = live_seq(a, t, sh);
    if (seq[j] >= 0) {
      const float4* p = reinterpret_cast<const float4*>(a.logits) + 2 * t;
      const float4 u = __ldg(p), v = __ldg(p + 1);
      l[j][0] = u.x; l[j][1] = u.y; l[j][2] = u.z; l[j][3] = u.w;
      l[j][4] = v.x; l[j][5] = v.y; l[j][6] = v.z; l[j][7] = v.w;
    } else if (t < a.T && a.dlogits) {
      float4* p = reinterpret_cast<float4*>(a.dlogits) + 2 * t;
      p[0] = p[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  for (int w0 = first; w0 <= last; w0 += kWindow) {
    const int n = min(last - w0 + 1, kWindow);
    // the chunk's first and last sequence may run through many chunks: all threads sum their slots
    for (int k = 0; k < 2; ++k) {
      const int s = k == 0 ? first : last;
      if ((k == 1 && last == first) || s < w0 || s >= w0 + n) continue;
      const int q = threadIdx.x & (kSlot - 1), g = threadIdx.x / kSlot;
      sh.red[g][q] = q <= kE ? sum_slots(a, s, q, g, NT / kSlot) : 0;
      __syncthreads();
      if (threadIdx.x <= kE) {
        int v = 0;
        for (int i = 0; i < NT / kSlot; ++i) v += sh.red[i][threadIdx.x];
        sh.hist[s - w0][threadIdx.x] = v;
      }
      __syncthreads();
    }
    // the others lie in this chunk alone: one slot each
    for (int i = threadIdx.x; i < n * (kE + 1); i += NT) {
      const int s = w0 + i / (kE + 1), q = i % (kE + 1);
      if (s != first && s != last) sh.hist[s - w0][q] = sum_slots(a, s, q, 0, 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
      const int s = w0 + i;
      if (bound_of(a, s) < bound_of(a, s + 1) && owner_of(a, s) == c)
        for (int e = 0; e < kE; ++e) a.counts[(int64_t)s * kE + e] = sh.hist[i][e];
      const int live = sh.hist[i][kE];
      const float half = live > 0 ? 0.5f / (float)live : 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) sh.hist[i][e] = __float_as_int((float)sh.hist[i][e] * half);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const int s = seq[j] - w0;
      if (seq[j] < 0 || s < 0 || s >= n) continue;
      float top = l[j][0];
#pragma unroll
      for (int e = 1; e < kE; ++e) top = fmaxf(top, l[j][e]);
      float p[kE], f[kE], total = 0.f, dot = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        p[e] = expf(l[j][e] - top);
        total += p[e];
        f[e] = __int_as_float(sh.hist[s][e]);
      }
      const float inv = 1.0f / total;
      const float lse = top + logf(total);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        p[e] *= inv;
        dot = fmaf(f[e], p[e], dot);
      }
      sum_f += dot;
      sum_z = fmaf(lse, lse, sum_z);
      if (a.dlogits) {
        const float ka = a.a * (float)kE * inv_n, kb = 2.0f * a.b * inv_n * lse;
#pragma unroll
        for (int e = 0; e < kE; ++e) p[e] *= fmaf(ka, f[e] - dot, kb);
        float4* o = reinterpret_cast<float4*>(a.dlogits) + 2 * ((int64_t)c * kChunk + j * NT + threadIdx.x);
        o[0] = make_float4(p[0], p[1], p[2], p[3]);
        o[1] = make_float4(p[4], p[5], p[6], p[7]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum_f += __shfl_xor_sync(~0u, sum_f, o);
    sum_z += __shfl_xor_sync(~0u, sum_z, o);
  }
  if ((threadIdx.x & 31) == 0) sh.fred[threadIdx.x >> 5] = make_float2(sum_f, sum_z);
  __syncthreads();
  if (threadIdx.x == 0) {
    float2 s = sh.fred[0];
    for (int w = 1; w < NT / 32; ++w) {
      s.x += sh.fred[w].x;
      s.y += sh.fred[w].y;
    }
    a.chunk_sum[c] = s;
  }
}

// Zero counts of the empty sequences, shared out over `parts` blocks.
template <int NT>
__device__ __forceinline__ void empty_counts(const BalanceArgs& a, int part, int parts) {
  for (int64_t s = (int64_t)part * NT + threadIdx.x; s < a.n_seq; s += (int64_t)parts * NT) {
    if (a.seq) {
      const int64_t lo = __ldg(a.seq + s), hi = __ldg(a.seq + s + 1);
      if (lo > hi || (s == 0 && lo < 0) || (s == a.n_seq - 1 && hi > a.T)) flag_error(a.err, MOE_DEVERR_OFFSETS);
    }
    if (bound_of(a, (int)s) >= bound_of(a, (int)s + 1)) {
      int4* o = reinterpret_cast<int4*>(a.counts + s * kE);
      o[0] = o[1] = make_int4(0, 0, 0, 0);
    }
  }
}

// N, the live tokens of all chunks, by all threads of a block.
template <int NT>
__device__ __forceinline__ int64_t total_live(const BalanceArgs& a, Shared<NT>& sh) {
  int v = 0;
  for (int c = threadIdx.x; c < a.n_chunks; c += NT) v += __ldcg(a.chunk_live + c);
  v = __reduce_add_sync(~0u, v);
  if ((threadIdx.x & 31) == 0) sh.ired[threadIdx.x >> 5] = v;
  __syncthreads();
  int n = 0;
  for (int w = 0; w < NT / 32; ++w) n += sh.ired[w];
  __syncthreads();
  return n;
}

// The losses from the chunks' sums, in double and in a fixed order, by one block.
template <int NT>
__device__ __forceinline__ void write_loss(const BalanceArgs& a, int64_t n, Shared<NT>& sh) {
  double f = 0.0, z = 0.0;
  for (int c = threadIdx.x; c < a.n_chunks; c += NT) {
    const float2 v = __ldcg(a.chunk_sum + c);
    f += (double)v.x;
    z += (double)v.y;
  }
  double2* red = reinterpret_cast<double2*>(&sh.hist[0][0]);
  red[threadIdx.x] = make_double2(f, z);
  __syncthreads();
  for (int w = NT / 2; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) {
      red[threadIdx.x].x += red[threadIdx.x + w].x;
      red[threadIdx.x].y += red[threadIdx.x + w].y;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double inv = n > 0 ? 1.0 / (double)n : 0.0;
    const double balance = (double)kE * red[0].x * inv, zl = red[0].y * inv;
    a.loss[0] = (float)((double)a.a * balance + (double)a.b * zl);
    a.loss[1] = (float)balance;
    a.loss[2] = (float)zl;
  }
}

template <int NT>
__global__ void __launch_bounds__(NT) balance_count_kernel(const BalanceArgs a) {
  __shared__ __align__(16) Shared<NT> sh;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  empty_counts<NT>(a, blockIdx.x, gridDim.x);
  for (int c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    count_chunk<NT>(a, c, sh);
    __syncthreads();
  }
}

template <int NT>
__global__ void __launch_bounds__(NT) balance_gradient_kernel(const BalanceArgs a) {
  __shared__ __align__(16) Shared<NT> sh;
  pdl_wait();
  const int64_t n = total_live<NT>(a, sh);
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
  for (int c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    gradient_chunk<NT>(a, c, inv_n, sh);
    __syncthreads();
  }
  // the block that finishes last adds up the chunks' sums
  if (threadIdx.x == 0) {
    __threadfence();
    sh.done = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (sh.done) write_loss<NT>(a, n, sh);
}

}  // namespace

int64_t balance_slot_bytes(int64_t T, int64_t n_seq) {
  const int64_t chunks = T > 0 ? (T + kChunk - 1) / kChunk : 1;
  return (chunks + n_seq) * kSlot * 4 + chunks * 16 + 64;
}

cudaError_t launch_balance(const moe_config_t& c, const float* logits, const int32_t* idx, const uint8_t* mask,
                           const int32_t* seq, int32_t n_seq, float coef_a, float coef_b, int32_t* counts, float* loss,
                           float* dlogits, void* ws, cudaStream_t s, const Ctx& ctx) {
  BalanceArgs a = {};
  a.logits = logits;
  a.idx = idx;
  a.mask = mask;
  a.seq = seq;
  a.T = c.T;
  a.n_seq = n_seq;
  a.n_chunks = c.T > 0 ? (int32_t)((c.T + kChunk - 1) / kChunk) : 1;
  a.a = coef_a;
  a.b = coef_b;
  a.counts = counts;
  a.loss = loss;
  a.dlogits = dlogits;
  a.slots = static_cast<int32_t*>(ws);
  a.chunk_sum = reinterpret_cast<float2*>(a.slots + ((int64_t)a.n_chunks + n_seq) * kSlot);
  a.chunk_live = reinterpret_cast<int32_t*>(a.chunk_sum + a.n_chunks);
  a.ticket = a.chunk_live + a.n_chunks;
  a.err = ctx.err;
  const int cap = ctx.num_sms * 4;
  const int grid = a.n_chunks < cap ? a.n_chunks : cap;
  cudaError_t e = launch_pdl(balance_count_kernel<256>, dim3(grid), dim3(256), 0, s, no_extra_attr(), a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(balance_gradient_kernel<256>, dim3(grid), dim3(256), 0, s, no_extra_attr(), a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_loss_workspace_size(const moe_config_t* cfg, int32_t n_seq) {
  if (validate_config(cfg) != MOE_OK || n_seq < 1 || n_seq > MOE_BALANCE_MAX_SEQS) return 0;
  return (size_t)((balance_slot_bytes(cfg->T, n_seq) + 255) & ~(int64_t)255);
}

moe_status_t moe_balance_loss(const moe_config_t* cfg, const float* logits, const int32_t* topk_idx,
                              const uint8_t* token_mask, const int32_t* seq_offsets, int32_t n_seq,
                              float balance_coef, float z_coef, int32_t* counts, float* loss, float* dlogits, void* ws,
                              size_t ws_bytes, moe_stream_t stream) {
  Range range_("moe_balance_loss");
  moe_status_t st = validate_config(cfg);
  if (st != MOE_OK) return st;
  auto bad16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; };
  if (n_seq < 1 || n_seq > MOE_BALANCE_MAX_SEQS || (!seq_offsets && n_seq != 1)) return MOE_ERR_INVALID_ARG;
  if (!isfinite(balance_coef) || !isfinite(z_coef)) return MOE_ERR_INVALID_ARG;
  if (!counts || !loss || bad16(counts) || bad16(loss)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!logits || !topk_idx)) return MOE_ERR_INVALID_ARG;
  if (bad16(logits) || bad16(topk_idx) || bad16(dlogits) || (reinterpret_cast<uintptr_t>(seq_offsets) & 3u))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_balance_loss_workspace_size(cfg, n_seq)) return MOE_ERR_WORKSPACE;
  if (bad16(ws)) return MOE_ERR_INVALID_ARG;
  Ctx ctx;
  if ((st = current_ctx(ctx)) != MOE_OK) return st;
  const cudaError_t e = launch_balance(*cfg, logits, topk_idx, token_mask, seq_offsets, n_seq, balance_coef, z_coef,
                                       counts, loss, dlogits, ws, stream, ctx);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
