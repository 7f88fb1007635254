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
// Three forms, each a chain of dependent steps, which is what bounds them up to
// about 10^5 tokens (a launch adds 2 to 3 us, a round trip to L2 0.5 us):
//   one chunk of 1024 tokens: one block, everything in shared memory;
//   up to 16 chunks: one cluster, a block a chunk that keeps its logits in
//     registers across the cluster's barrier.  The pairs (chunk c, sequence s)
//     that meet form a staircase, each step of which raises c or s, so c + s
//     names a slot of its own for the pair's counts;
//   more: cleared totals per sequence, a kernel that adds the chunks' counts to
//     them, a kernel for the rest.
// Measured: 3.7 us for 32 tokens, 10.3 us for 16384 (64 sequences), 1.6 + 11.8 +
// 25.0 us for 2^20 (1000 sequences), of which 11.7 us are its 76 MB at the copy
// rate: there a chunk's chain, three blocks an SM and three rounds, bounds it.
// Counts are integers, so no order matters; the float sums run in a fixed order
// (thread, warp, chunk), so results do not depend on scheduling.
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kE = 8;
constexpr int kNT = 512;       // threads of a block
constexpr int kChunk = 1024;   // tokens of a chunk
constexpr int kTok = kChunk / kNT;
constexpr int kWindow = 1024;  // sequences held at once (a chunk meets more only if most are empty)
constexpr int kSlot = 16;      // int32 of a slot: 8 counts, live tokens, padding to 64 bytes
constexpr int kCluster = 16;   // most blocks of the cluster form

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
  int32_t* slots;              // cluster: [n_chunks + n_seq][kSlot];  totals: [n_seq][kSlot]
  int32_t* chunk_live;         // cluster: [n_chunks]
  float2* chunk_sum;           // [n_chunks]: sum of sum_e f p, sum of lse^2
  int32_t* ticket;             // [0]: blocks of pass 2 that are done, [1]: live tokens
  int* err;
};

__device__ __forceinline__ int bound_of(const BalanceArgs& a, int s) {
  const int T = (int)a.T;  // at most 2^24
  const int v = a.seq ? __ldg(a.seq + s) : (s == 0 ? 0 : T);
  return min(max(v, 0), T);
}

struct __align__(16) Shared {
  int hist[kWindow][kE + 1];  // pass 1: counts and live tokens; pass 2: f (as float bits) in [0, E)
  int bound[kWindow + 1];     // offsets of the window's sequences
  float2 fred[kNT / 32];
  unsigned found[kNT / 32];
  int ired[kNT / 32];
  int done;
};

// A chunk of tokens and the sequences that they can belong to.
struct Chunk {
  int first, last;   // last < first: none
  int t0;            // first token
  bool live[kTok];   // unmasked, inside the range of all sequences
};
constexpr int kScan = 8;  // offsets a thread looks at in the one-round search

// Sequences that end at or before token t, by the whole block: every round
// tests kNT evenly spaced ones at once (empty sequences are passed over, so this
// is the sequence of t when t lies in one).
__device__ __forceinline__ int block_seq_of(const BalanceArgs& a, int t) {
  int lo = 0, hi = a.n_seq;
  while (lo < hi) {
    const int step = (hi - lo + kNT - 1) / kNT;
    const int64_t s = lo + (int64_t)threadIdx.x * step;
    const int c = __syncthreads_count(s < hi && bound_of(a, (int)s + 1) <= t);
    if (step == 1) return lo + c;
    if (c == 0) return lo;
    const int64_t next = lo + (int64_t)c * step;
    lo += (c - 1) * step + 1;
    if (next < hi) hi = (int)next;
  }
  return lo;
}

// Sequences that end at or before t0 and t1, in one round for up to kNT * kScan
// sequences: every thread looks at kScan neighbouring offsets.
__device__ __forceinline__ int2 block_seqs_of(const BalanceArgs& a, int t0, int t1, Shared& sh) {
  if (a.n_seq > kNT * kScan) return make_int2(block_seq_of(a, t0), block_seq_of(a, t1));
  int c0 = 0, c1 = 0;
  for (int s = threadIdx.x; s < a.n_seq; s += kNT) {
    const int v = bound_of(a, s + 1);
    c0 += v <= t0;
    c1 += v <= t1;
  }
  // at most 4096 in all: both in one word.  sh.found is next written a chunk
  // later, behind other barriers
  const unsigned both = __reduce_add_sync(~0u, (unsigned)c0 | (unsigned)c1 << 16);
  if ((threadIdx.x & 31) == 0) sh.found[threadIdx.x >> 5] = both;
  __syncthreads();
  unsigned sum = 0;
#pragma unroll
  for (int w = 0; w < kNT / 32; ++w) sum += sh.found[w];
  return make_int2((int)(sum & 0xffffu), (int)(sum >> 16));
}

__device__ __forceinline__ Chunk open_chunk(const BalanceArgs& a, int c, const uint8_t (&mask)[kTok], Shared& sh) {
  Chunk k;
  k.t0 = c * kChunk;
  const int begin = bound_of(a, 0), end = bound_of(a, a.n_seq);
  int64_t t1 = (int64_t)k.t0 + kChunk;
  if (t1 > end) t1 = end;
  const int t0 = k.t0 > begin ? k.t0 : begin;
  k.first = 0;
  k.last = -1;
  if (t0 < t1) {
    const int2 s = a.n_seq == 1 ? make_int2(0, 0) : block_seqs_of(a, t0, (int)t1 - 1, sh);
    k.first = s.x < a.n_seq ? s.x : a.n_seq - 1;
    k.last = s.y < a.n_seq ? s.y : a.n_seq - 1;
  }
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const int64_t t = (int64_t)k.t0 + j * kNT + threadIdx.x;
    k.live[j] = mask[j] && t >= begin && t < end;
  }
  return k;
}

// Window of n sequences from w0 on: offsets to shared memory, and for each of
// the thread's live tokens its sequence relative to w0, or -1.
__device__ __forceinline__ void open_window(const BalanceArgs& a, const Chunk& k, int w0, int n, int (&seq)[kTok],
                                            Shared& sh) {
  for (int i = threadIdx.x; i <= n; i += kNT) sh.bound[i] = bound_of(a, w0 + i);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const int t = k.t0 + j * kNT + (int)threadIdx.x;
    seq[j] = -1;
    if (k.live[j] && t >= sh.bound[0] && t < sh.bound[n]) {
      int lo = 0, hi = n - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sh.bound[mid + 1] <= t)
          lo = mid + 1;
        else
          hi = mid;
      }
      seq[j] = lo;
    }
  }
}

// Drops the choices of tokens that are not live; the chunk's live tokens (in every thread).
__device__ __forceinline__ int live_choices(const BalanceArgs& a, const Chunk& k, int2 (&e)[kTok], Shared& sh) {
  int live = 0;
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    if (k.live[j]) {
      if ((unsigned)e[j].x >= kE || (unsigned)e[j].y >= kE) flag_error(a.err, MOE_DEVERR_EXPERT_INDEX);
      ++live;
    } else {
      e[j] = make_int2(-1, -1);
    }
  }
  live = __reduce_add_sync(~0u, live);
  if ((threadIdx.x & 31) == 0) sh.ired[threadIdx.x >> 5] = live;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kNT / 32; ++w) sum += sh.ired[w];
  return sum;  // sh.ired is next written after a barrier of count_window
}

// Counts and live tokens of the n sequences from w0 on, into sh.hist.
__device__ __forceinline__ void count_window(const BalanceArgs& a, const Chunk& k, int w0, int n, const int2 (&e)[kTok],
                                             int (&seq)[kTok], Shared& sh) {
  for (int i = threadIdx.x; i < n * (kE + 1); i += kNT) (&sh.hist[0][0])[i] = 0;
  open_window(a, k, w0, n, seq, sh);  // its barrier also covers the zeros
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    // 32 neighbouring tokens mostly lie in one sequence: then the warp adds up
    // eight one-byte counts in two words (64 at most in a byte) and nine lanes add
    // them to the sequence's, where all lanes would queue at the same words
    const unsigned live = __ballot_sync(~0u, seq[j] >= 0);
    if (live == 0) continue;
    const int s0 = __shfl_sync(~0u, seq[j], __ffs(live) - 1);
    if (__all_sync(~0u, seq[j] < 0 || seq[j] == s0)) {
      unsigned long long v = 0;
      if (seq[j] >= 0) {
        if ((unsigned)e[j].x < kE) v += 1ull << (8 * e[j].x);
        if ((unsigned)e[j].y < kE) v += 1ull << (8 * e[j].y);
      }
      const unsigned lo = __reduce_add_sync(~0u, (unsigned)v), hi = __reduce_add_sync(~0u, (unsigned)(v >> 32));
      const int lane = threadIdx.x & 31;
      if (lane <= kE) {
        const int mine = lane == kE ? __popc(live) : (int)(((lane < 4 ? lo : hi) >> (8 * (lane & 3))) & 0xffu);
        if (mine) atomicAdd(&sh.hist[s0][lane], mine);
      }
    } else if (seq[j] >= 0) {
      if ((unsigned)e[j].x < kE) atomicAdd(&sh.hist[seq[j]][e[j].x], 1);
      if ((unsigned)e[j].y < kE) atomicAdd(&sh.hist[seq[j]][e[j].y], 1);
      atomicAdd(&sh.hist[seq[j]][kE], 1);
    }
  }
  __syncthreads();
}

// A chunk's masks, choices and logits, asked for before it is known which tokens
// are live (a padded row's values are dropped), so that they travel during the
// search (the counts: while the block works on the chunk before).
__device__ __forceinline__ void load_masks(const BalanceArgs& a, int c, uint8_t (&mask)[kTok]) {
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const int64_t t = (int64_t)c * kChunk + j * kNT + threadIdx.x;
    mask[j] = t < a.T ? (a.mask ? __ldg(a.mask + t) : 1) : 0;
  }
}
__device__ __forceinline__ void load_choices(const BalanceArgs& a, int c, int2 (&e)[kTok]) {
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const int64_t t = (int64_t)c * kChunk + j * kNT + threadIdx.x;
    if (t < a.T) e[j] = __ldg(reinterpret_cast<const int2*>(a.idx) + t);
  }
}
__device__ __forceinline__ void load_logits(const BalanceArgs& a, int c, float (&l)[kTok][kE]) {
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const int64_t t = (int64_t)c * kChunk + j * kNT + threadIdx.x;
    if (t < a.T) {
      const float4* p = reinterpret_cast<const float4*>(a.logits) + 2 * t;
      const float4 u = __ldcs(p), v = __ldcs(p + 1);
      l[j][0] = u.x; l[j][1] = u.y; l[j][2] = u.z; l[j][3] = u.w;
      l[j][4] = v.x; l[j][5] = v.y; l[j][6] = v.z; l[j][7] = v.w;
    }
  }
}

// dlogits 0 for the chunk's tokens that are not live.
__device__ __forceinline__ void clear_dead(const BalanceArgs& a, const Chunk& k) {
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const int64_t t = (int64_t)k.t0 + j * kNT + threadIdx.x;
    if (!k.live[j] && t < a.T && a.dlogits) {
      float4* p = reinterpret_cast<float4*>(a.dlogits) + 2 * t;
      p[0] = p[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

// sh.hist of the window, now the sequences' totals, to f (as float bits); the
// chunk that holds a sequence's first token writes its counts.
__device__ __forceinline__ void counts_to_f(const BalanceArgs& a, int c, int w0, int n, Shared& sh) {
  for (int i = threadIdx.x; i < n; i += kNT) {
    if (sh.bound[i] < sh.bound[i + 1] && sh.bound[i] / kChunk == c) {
      int4* o = reinterpret_cast<int4*>(a.counts + ((int64_t)w0 + i) * kE);
      o[0] = make_int4(sh.hist[i][0], sh.hist[i][1], sh.hist[i][2], sh.hist[i][3]);
      o[1] = make_int4(sh.hist[i][4], sh.hist[i][5], sh.hist[i][6], sh.hist[i][7]);
    }
    const int live = sh.hist[i][kE];
    const float half = live > 0 ? 0.5f / (float)live : 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) sh.hist[i][e] = __float_as_int((float)sh.hist[i][e] * half);
  }
  __syncthreads();
}

// The window's tokens: gradients, and their part of the two sums.
__device__ __forceinline__ void window_tokens(const BalanceArgs& a, const Chunk& k, const float (&l)[kTok][kE],
                                              const int (&seq)[kTok], float inv_n, float2& sum, const Shared& sh) {
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    if (seq[j] < 0) continue;
    float top = l[j][0];
#pragma unroll
    for (int e = 1; e < kE; ++e) top = fmaxf(top, l[j][e]);
    float p[kE], f[kE], total = 0.f, dot = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      // within 2 + 1.2 |l - top| ulp, the logarithm and quotient below within 3 (expf and
      // logf, within 2 and 1, spill here: 47 against 39 us a call at 2^20 tokens)
      p[e] = __expf(l[j][e] - top);
      total += p[e];
      f[e] = __int_as_float(sh.hist[seq[j]][e]);
    }
    const float inv = __fdividef(1.0f, total);
    const float lse = top + __logf(total);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      p[e] *= inv;
      dot = fmaf(f[e], p[e], dot);
    }
    sum.x += dot;
    sum.y = fmaf(lse, lse, sum.y);
    if (a.dlogits) {
      const float ka = a.a * (float)kE * inv_n, kb = 2.0f * a.b * inv_n * lse;
#pragma unroll
      for (int e = 0; e < kE; ++e) p[e] *= fmaf(ka, f[e] - dot, kb);
      float4* o = reinterpret_cast<float4*>(a.dlogits) + 2 * ((int64_t)k.t0 + j * kNT + threadIdx.x);
      o[0] = make_float4(p[0], p[1], p[2], p[3]);
      o[1] = make_float4(p[4], p[5], p[6], p[7]);
    }
  }
}

// The block's sum, in thread 0, which reads sh.fred behind the barrier: a barrier
// between two calls keeps the second one's writes behind these reads.
__device__ __forceinline__ float2 block_sum(float2 s, Shared& sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.x += __shfl_xor_sync(~0u, s.x, o);
    s.y += __shfl_xor_sync(~0u, s.y, o);
  }
  if ((threadIdx.x & 31) == 0) sh.fred[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = sh.fred[0];
    for (int w = 1; w < kNT / 32; ++w) {
      s.x += sh.fred[w].x;
      s.y += sh.fred[w].y;
    }
  }
  return s;
}

// Zero counts of the empty sequences and the check of the offsets, shared out over `parts` blocks.
__device__ __forceinline__ void empty_counts(const BalanceArgs& a, int part, int parts) {
  for (int64_t s = (int64_t)part * kNT + threadIdx.x; s < a.n_seq; s += (int64_t)parts * kNT) {
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

__device__ __forceinline__ void store_loss(const BalanceArgs& a, double f, double z, int n) {
  const double inv = n > 0 ? 1.0 / (double)n : 0.0;
  const double balance = (double)kE * f * inv, zl = z * inv;
  // a term without weight stays out, an infinite one too
  a.loss[0] = (float)((a.a != 0.f ? (double)a.a * balance : 0.0) + (a.b != 0.f ? (double)a.b * zl : 0.0));
  a.loss[1] = (float)balance;
  a.loss[2] = (float)zl;
}

// The losses from the chunks' sums, in double and in a fixed order, by one block.
__device__ __forceinline__ void write_loss(const BalanceArgs& a, int n, Shared& sh) {
  double f = 0.0, z = 0.0;
  for (int c = threadIdx.x; c < a.n_chunks; c += kNT) {
    const float2 v = __ldcg(a.chunk_sum + c);
    f += (double)v.x;
    z += (double)v.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    f += __shfl_xor_sync(~0u, f, o);
    z += __shfl_xor_sync(~0u, z, o);
  }
  double2* red = reinterpret_cast<double2*>(&sh.hist[0][0]);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_double2(f, z);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kNT / 32; ++w) {
      f += red[w].x;
      z += red[w].y;
    }
    store_loss(a, f, z, n);
  }
}

// One chunk: counts, f, gradients and losses in one block.
__global__ void __launch_bounds__(kNT, 1) balance_single_kernel(const BalanceArgs a) {
  __shared__ Shared sh;
  pdl_wait();
  float l[kTok][kE];
  int2 e[kTok];
  uint8_t mask[kTok];
  load_masks(a, 0, mask);
  load_logits(a, 0, l);
  load_choices(a, 0, e);
  const Chunk k = open_chunk(a, 0, mask, sh);
  empty_counts(a, 0, 1);
  clear_dead(a, k);
  const int n = live_choices(a, k, e, sh);
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
  float2 sum = make_float2(0.f, 0.f);
  for (int w0 = k.first; w0 <= k.last; w0 += kWindow) {
    const int m = min(k.last - w0 + 1, kWindow);
    int seq[kTok];
    count_window(a, k, w0, m, e, seq, sh);
    counts_to_f(a, 0, w0, m, sh);
    window_tokens(a, k, l, seq, inv_n, sum, sh);
    __syncthreads();
  }
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) store_loss(a, (double)sum.x, (double)sum.y, n);
}

__global__ void __launch_bounds__(kNT, 1) balance_cluster_kernel(const BalanceArgs a) {
  __shared__ Shared sh;
  pdl_wait();
  const int c = blockIdx.x;
  float l[kTok][kE];
  int2 e[kTok];
  uint8_t mask[kTok];
  load_masks(a, c, mask);
  load_logits(a, c, l);
  load_choices(a, c, e);
  const Chunk k = open_chunk(a, c, mask, sh);
  empty_counts(a, c, gridDim.x);
  const int mine = live_choices(a, k, e, sh);
  int seq[kTok];
  for (int w0 = k.first; w0 <= k.last; w0 += kWindow) {
    const int m = min(k.last - w0 + 1, kWindow);
    count_window(a, k, w0, m, e, seq, sh);
    for (int i = threadIdx.x; i < m * (kE + 1); i += kNT) {
      const int s = i / (kE + 1), q = i - s * (kE + 1);
      a.slots[((int64_t)c + w0 + s) * kSlot + q] = sh.hist[s][q];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) a.chunk_live[c] = mine;
  ptx::cluster_sync();  // the slots and live tokens of all chunks are written
  int n = 0;
#pragma unroll
  for (int i = 0; i < kCluster; ++i)
    if (i < a.n_chunks) n += __ldcg(a.chunk_live + i);
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
  clear_dead(a, k);
  float2 sum = make_float2(0.f, 0.f);
  const bool same = k.last - k.first < kWindow;  // seq and sh.bound still hold the only window
  for (int w0 = k.first; w0 <= k.last; w0 += kWindow) {
    const int m = min(k.last - w0 + 1, kWindow);
    if (!same) open_window(a, k, w0, m, seq, sh);
    // a sequence's slots: one for each chunk that it meets
    for (int i = threadIdx.x; i < m * (kE + 1); i += kNT) {
      const int s = i / (kE + 1), q = i - s * (kE + 1);
      const int lo = sh.bound[s], hi = sh.bound[s + 1];
      const int c0 = lo / kChunk, c1 = lo < hi ? (hi - 1) / kChunk : -1;
      int v = 0;
#pragma unroll
      for (int j = 0; j < kCluster; ++j)
        if (j >= c0 && j <= c1 && j < a.n_chunks) v += __ldcg(a.slots + ((int64_t)j + w0 + s) * kSlot + q);
      sh.hist[s][q] = v;
    }
    __syncthreads();
    counts_to_f(a, c, w0, m, sh);
    window_tokens(a, k, l, seq, inv_n, sum, sh);
    __syncthreads();
  }
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) a.chunk_sum[c] = sum;
  ptx::cluster_sync();  // the chunks' sums are written
  if (c == 0) write_loss(a, n, sh);
}

__global__ void __launch_bounds__(kNT, 3) balance_count_kernel(const BalanceArgs a) {
  __shared__ Shared sh;
  pdl_wait();
  empty_counts(a, blockIdx.x, gridDim.x);
  uint8_t mask[kTok];
  int2 next[kTok];
  load_masks(a, blockIdx.x, mask);
  load_choices(a, blockIdx.x, next);
  for (int c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    const Chunk k = open_chunk(a, c, mask, sh);
    int2 e[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j) e[j] = next[j];
    if (c + (int)gridDim.x < a.n_chunks) {
      load_masks(a, c + gridDim.x, mask);
      load_choices(a, c + gridDim.x, next);
    }
    const int live = live_choices(a, k, e, sh);
    if (threadIdx.x == 0) atomicAdd(a.ticket + 1, live);
    for (int w0 = k.first; w0 <= k.last; w0 += kWindow) {
      const int m = min(k.last - w0 + 1, kWindow);
      int seq[kTok];
      count_window(a, k, w0, m, e, seq, sh);
      for (int i = threadIdx.x; i < m * (kE + 1); i += kNT) {
        const int s = i / (kE + 1), q = i - s * (kE + 1), v = sh.hist[s][q];
        if (v) atomicAdd(a.slots + ((int64_t)w0 + s) * kSlot + q, v);
      }
      __syncthreads();
    }
    if (k.last < k.first) __syncthreads();  // no window's barriers before sh.ired is written again
  }
}

__global__ void __launch_bounds__(kNT, 3) balance_gradient_kernel(const BalanceArgs a) {
  __shared__ Shared sh;
  pdl_wait();
  const int n = __ldcg(a.ticket + 1);
  const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
  uint8_t mask[kTok];
  load_masks(a, blockIdx.x, mask);
  for (int c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    const Chunk k = open_chunk(a, c, mask, sh);
    float l[kTok][kE];  // after the search: across it they cost a block's registers or spill
    load_logits(a, c, l);
    if (c + (int)gridDim.x < a.n_chunks) load_masks(a, c + gridDim.x, mask);
    clear_dead(a, k);
    float2 sum = make_float2(0.f, 0.f);
    for (int w0 = k.first; w0 <= k.last; w0 += kWindow) {
      const int m = min(k.last - w0 + 1, kWindow);
      for (int i = threadIdx.x; i < m * 3; i += kNT) {
        const int s = i / 3, q = i - s * 3;
        const int4 v = __ldcg(reinterpret_cast<const int4*>(a.slots + ((int64_t)w0 + s) * kSlot) + q);
        int* h = &sh.hist[s][4 * q];
        h[0] = v.x;
        if (q < 2) {
          h[1] = v.y;
          h[2] = v.z;
          h[3] = v.w;
        }
      }
      int seq[kTok];
      open_window(a, k, w0, m, seq, sh);  // its barrier also covers the totals
      counts_to_f(a, c, w0, m, sh);
      window_tokens(a, k, l, seq, inv_n, sum, sh);
      if (w0 + kWindow <= k.last) __syncthreads();
    }
    // a chunk without a window (padding) has passed no barrier since the last chunk's sum was read
    if (k.last < k.first) __syncthreads();
    sum = block_sum(sum, sh);  // its barrier ends the use of sh.hist
    if (threadIdx.x == 0) a.chunk_sum[c] = sum;
  }
  // the block that finishes last adds up the chunks' sums
  if (threadIdx.x == 0) {
    __threadfence();
    sh.done = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (sh.done) write_loss(a, n, sh);
}

// Blocks that one cluster can have on this device: kCluster where 16 are
// accepted (a form beyond the portable 8), asked once per device.
int cluster_limit(const Ctx& ctx) {
  static std::atomic<int> cached[64];
  const int slot = ctx.dev >= 0 && ctx.dev < 64 ? ctx.dev : 0;
  int n = cached[slot].load(std::memory_order_relaxed);
  if (n > 0) return n;
  n = 8;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kNT);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int fit = 0;
  if (cudaFuncSetAttribute(balance_cluster_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&fit, balance_cluster_kernel, &cfg) == cudaSuccess && fit > 0)
    n = kCluster;
  (void)cudaGetLastError();
  cached[slot].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace

int64_t balance_slot_bytes(int64_t T, int64_t n_seq) {
  const int64_t chunks = (T + kChunk - 1) / kChunk;
  if (chunks <= 1) return 0;  // all in shared memory
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
  a.ticket = static_cast<int32_t*>(ws);  // 64 bytes
  a.slots = a.ticket + 16;
  a.chunk_sum = reinterpret_cast<float2*>(a.slots + ((int64_t)a.n_chunks + n_seq) * kSlot);
  a.chunk_live = reinterpret_cast<int32_t*>(a.chunk_sum + a.n_chunks);
  a.err = ctx.err;
  cudaError_t e;
  if (a.n_chunks == 1) {
    e = launch_pdl(balance_single_kernel, dim3(1), dim3(kNT), 0, s, no_extra_attr(), a);
  } else if (a.n_chunks <= cluster_limit(ctx)) {
    if (a.n_chunks > 8) {
      e = cudaFuncSetAttribute(balance_cluster_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute cl = {};
    cl.id = cudaLaunchAttributeClusterDimension;
    cl.val.clusterDim.x = (unsigned)a.n_chunks;
    cl.val.clusterDim.y = cl.val.clusterDim.z = 1;
    e = launch_pdl(balance_cluster_kernel, dim3(a.n_chunks), dim3(kNT), 0, s, cl, a);
  } else {
    e = cudaMemsetAsync(ws, 0, (size_t)(16 + (int64_t)n_seq * kSlot) * 4, s);
    if (e != cudaSuccess) return e;
    const int resident = ctx.num_sms * 3;
    const dim3 grid(a.n_chunks < resident ? a.n_chunks : resident);
    e = launch_pdl(balance_count_kernel, grid, dim3(kNT), 0, s, no_extra_attr(), a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(balance_gradient_kernel, grid, dim3(kNT), 0, s, no_extra_attr(), a);
  }
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
  const size_t need = moe_balance_loss_workspace_size(cfg, n_seq);
  if (ws_bytes < need || (need > 0 && !ws)) return MOE_ERR_WORKSPACE;
  if (bad16(ws)) return MOE_ERR_INVALID_ARG;
  Ctx ctx;
  if ((st = current_ctx(ctx)) != MOE_OK) return st;
  const cudaError_t e = launch_balance(*cfg, logits, topk_idx, token_mask, seq_offsets, n_seq, balance_coef, z_coef,
                                       counts, loss, dlogits, ws, stream, ctx);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
