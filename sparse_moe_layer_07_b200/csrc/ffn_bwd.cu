// Backward of the expert FFNs on the tcgen05 tensor cores (training).
//
// The pages give the forward pass only ("How does Grok-1 use a
// mixture-of-experts design?", sections "Expert implementation: SwiGLU at
// scale" and "Expert parallelism vs. tensor parallelism"); training
// differentiates that forward with the routing decisions held fixed.  For
// the kept rows r of expert e (token t = perm[r], weight w = row_scale[r]),
// with G = X W_gate, U = X W_up, H = silu(G) * U saved by the forward:
//   kDH : dHu[r, :] = dout[t, :] W_down[e]^T        (A = dout rows, B = W_down K-major)
//         epilogue: dH = w * dHu,  dG = dH * U * silu'(G),  dU = dH * silu(G),
//         and per-tile partials of <dHu, H> (= the routing weight's gradient
//         <dout, y>), summed later in a fixed order
//   kDX : dx[t, :] += dG[r, :] W_gate[e]^T + dU[r, :] W_up[e]^T
//         (K runs over both halves; B = W_gate / W_up read K-major straight from
//         their [E, d, f] layout; the epilogue adds into an fp32 sum by token:
//         two terms per token, so the order of the adds does not matter)
//   kWG : dW[e] = A_e^T B_e over the rows of expert e  (A, B MN-major:
//         dW_down = H^T (w * dout),  dW_gate = X^T dG,  dW_up = X^T dU); K is
//         the ragged row count: the expert's last K block issues only the
//         16-row MMA steps that hold its rows, and the rows of the last step
//         past the expert's end are zeroed in shared memory before the MMA
//         (by warp 6, which only kWG has).
// C8 variants (8-bit checkpoints): kDH decodes G and U from codes and bf16
// scales (2.1 bytes a value pair where bf16 G, U and H are 6), forms H again
// and writes hw = bf16(w * H), so that dW_down = hw^T dout takes dout as it is
// and the product w * dout is rounded nowhere; kWG writes bf16.  dG, dU and hw are
// rounded to bf16 in both pairs: the widest operands at this MMA rate (tf32 has
// half of it and twice the bytes).  A gradient is off by 0.0024 in the mean square
// for it, where its own rounding to bf16 alone makes 0.0017.  Measured
// (kDH / kDX / one of kWG's products): T 2048, d 1536, f 8192 119 / 202 / 105 us, where the
// products alone at the measured matrix rate are 63 / 126 / 63 and the operand
// tiles arrive from L2 at 11 to 12 TB/s; T 8192, d 6144, f 32768 5.3 / 10.9 / 5.5
// ms against 4.8 / 9.6 / 4.8 at the rate under the power limit.
// Pipeline as in ffn_tc.cu: persistent CTAs, warp 0 TMA, warp 1 MMA (lane 0
// alone) + TMEM (two 128 x 256 fp32 accumulators), warps 2-5 epilogue; every
// wait bounded.
#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kE = 8;
constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = 64;
// Epilogue warps: 4, one per TMEM lane quarter.  (The layout also allows 8, two
// per quarter each taking half of the tile's columns; for kDH that measured 14%
// slower than 4 relative to the forward GEMMs in the same capture.)
// C8 is 0, or with 8-bit checkpoints the number of kDH's epilogue warps: its
// epilogue decodes as well, and where the tile's products are few (8 clocks per
// unit of d) it is what the tile waits for.  8 warps against 4 (f 8192): d 1536,
// T 2048 122 against 139 us; d 2560, T 4096 326 against 321; d 4096 480 against
// 475, where the products hide it.
template <int MODE, int C8 = 0>
struct Warps {
  static constexpr int kEpi = MODE == 0 && C8 ? C8 : 4;
  // weight gradients: one more warp zeroes the rows past an expert's end in its
  // last K block, so the MMA warp does not stall on it
  static constexpr int kZeroWarp = MODE == 2 ? 2 + kEpi : -1;
  static constexpr int kThreads = 64 + 32 * kEpi + (MODE == 2 ? 32 : 0);
};
constexpr int kTmemCols = 512;
constexpr int kAccStride = 256;
constexpr int CHUNK = 64 * BK * 2;      // 8 KB: 64 x 64 bf16
constexpr int A_BYTES = 2 * CHUNK;      // 16 KB: 128 x 64
constexpr int B_BYTES = 4 * CHUNK;      // 32 KB: 256 x 64
constexpr int STAGE = A_BYTES + B_BYTES;
constexpr int kStages = 4;
// weight gradients: each epilogue warp stages 32 rows x 32 fp32 (4 KB, 128-byte
// swizzled) for a TMA tile store, double buffered
constexpr int OUT_STAGE = 32 * 32 * 4;
constexpr int OUT_BYTES = 4 * 2 * OUT_STAGE;
constexpr int SMEM_BYTES = 1024 + kStages * STAGE + OUT_BYTES + 256;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
// full, empty, zeroed (kStages each), tfull, tempty (2 each), drain, then the
// TMEM slot, the abort flag and the producer's stage count
static_assert((3 * kStages + 5) * 8 + 12 <= 256, "barrier area");

enum Mode { kDH = 0, kDX = 1, kWG = 2 };

struct WgShape {           // dW [E, M, N]
  int M, m_tiles, n_tiles; // M / BM, N / BN
  int m_outer;             // tiles of one expert ordered M-block major
};

struct BwdArgs {
  const int32_t* offsets;  // [E + 1]
  int64_t rows_alloc;      // rows of the grouped buffers
  int n_tiles;             // N / BN (kDX: d / bn)
  int bn;                  // kDX: columns of a tile, 256 or 192
  int num_kb;              // kDH: d / BK;  kDX: 2 f / BK
  int half_kb;             // kDX: f / BK (first half dG x W_gate, second dU x W_up)
  const int32_t* perm;     // kDX: token of each row
  int64_t n_tok;
  const float* row_scale;  // kDH
  const __nv_bfloat16* G;  // kDH inputs [rows, f]
  const __nv_bfloat16* U;
  const __nv_bfloat16* H;
  Codes8 codes;            // kDH, C8: instead of G, U, H
  __nv_bfloat16* hw;       // kDH, C8: output [rows, f]
  __nv_bfloat16* dG;       // kDH outputs [rows, f]
  __nv_bfloat16* dU;
  float* dw_part;          // kDH: [rows, n_tiles * parts per tile]
  float* out;              // kDX: dx32 [T, d];  kWG: dW [E, M, N]
  int64_t ld;              // kDH: f;  kDX: d
  WgShape wg[3];           // kWG: C8 all three products, else the first
  int* err;
};

// kWG, C8: operands and outputs of the second and third product beside tmA0 x
// tmB0 -> tmOut and tmA1 x tmB1.
struct WgMaps {
  CUtensorMap b2, out1, out2;
};
struct NoMaps {};
template <int MODE, int C8>
using MoreMaps = std::conditional_t<MODE == kWG && C8 != 0, WgMaps, NoMaps>;

struct Sched {
  int offs[kE + 1];
  int mt[kE];              // row blocks (kDH, kDX) of each expert
  int prefix[kE + 1];
};

struct Tile {
  int e, m0, rows, n0, nb;
  int part;                // kWG, C8: which of the three products
  int row0, nrows, nkb;    // kWG: the expert's grouped rows and K blocks
};

template <int MODE, int C8>
__device__ __forceinline__ Tile decode_tile(const Sched& s, const BwdArgs& a, int L) {
  Tile t;
  t.part = 0;
  if (MODE == kWG && C8) {  // the products have the same number of tiles
    t.part = (L >= s.prefix[kE]) + (L >= 2 * s.prefix[kE]);
    L -= t.part * s.prefix[kE];
  }
  int e = 0;
#pragma unroll
  for (int k = 1; k < kE; ++k)
    if (L >= s.prefix[k]) e = k;
  const int local = L - s.prefix[e];
  t.e = e;
  t.row0 = s.offs[e];
  t.nrows = s.offs[e + 1] - s.offs[e];
  if (MODE == kWG) {
    const WgShape& w = a.wg[t.part];
    int mb, nb;
    if (w.m_outer) {
      mb = local / w.n_tiles;
      nb = local - mb * w.n_tiles;
    } else {
      nb = local / w.m_tiles;
      mb = local - nb * w.m_tiles;
    }
    t.m0 = mb * BM;
    t.rows = BM;
    t.n0 = nb * BN;
    t.nb = nb;
    t.nkb = (t.nrows + BK - 1) / BK;
  } else {
    const int nb = local / s.mt[e];
    const int mi = local - nb * s.mt[e];
    t.m0 = s.offs[e] + mi * BM;
    const int left = s.offs[e + 1] - t.m0;
    t.rows = left < BM ? left : BM;
    t.n0 = nb * (MODE == kDX ? a.bn : BN);
    t.nb = nb;
    t.nkb = MODE == kDH ? a.num_kb : 2 * a.half_kb;
  }
  return t;
}

template <int MODE>
__device__ __forceinline__ void build_schedule(Sched& sched, const BwdArgs& args) {
  bool ok = true;
  int prev = 0;
  for (int k = 0; k <= kE; ++k) {
    const int v = args.offsets[k];
    sched.offs[k] = v;
    if (v < prev || (int64_t)v > args.rows_alloc) ok = false;
    prev = v;
  }
  if (sched.offs[0] < 0) ok = false;
  if (!ok)
    for (int k = 0; k <= kE; ++k) sched.offs[k] = 0;
  int acc = 0;
  for (int k = 0; k < kE; ++k) {
    const int n = sched.offs[k + 1] - sched.offs[k];
    sched.mt[k] = (n + BM - 1) / BM;
    sched.prefix[k] = acc;
    // weight gradients: every expert owns its M x N tiles (zero when it has no rows)
    acc += MODE == kWG ? (ok ? args.wg[0].m_tiles * args.wg[0].n_tiles : 0) : sched.mt[k] * args.n_tiles;
  }
  sched.prefix[kE] = acc;
  if (!ok) flag_error(args.err, MOE_DEVERR_OFFSETS);
}

__device__ __forceinline__ void unpack8_bf16(const uint4 q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <int MODE, int C8>
__global__ void __launch_bounds__(Warps<MODE, C8>::kThreads, 1)
    bwd_gemm_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                    const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                    const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ MoreMaps<MODE, C8> more,
                    const BwdArgs args) {
  constexpr int S = kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * A_BYTES;
  uint8_t* sOut = smem + S * STAGE;  // 1024-byte aligned: S * STAGE is a multiple of 1024
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * STAGE + OUT_BYTES);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* zeroed = drain + 1;  // kWG: stage s of a ragged last K block is zeroed and ready
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(zeroed + S);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // kWG: K blocks whose loads the producer has issued (the zeroing warp waits on
  // a stage's full barrier only once its loads are issued, so the barrier is at
  // that K block's phase and not at an earlier phase of the same parity)
  volatile uint32_t* issued_kb = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);
  __shared__ Sched sched;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *issued_kb = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&zeroed[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 32 * Warps<MODE, C8>::kEpi);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 1) {
    prefetch_tmap(&tmA0);
    prefetch_tmap(&tmB0);
    if (MODE == kDX || (MODE == kDH && C8)) {
      prefetch_tmap(&tmA1);
      prefetch_tmap(&tmB1);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  pdl_wait();
  if (warp == 2 && lane == 0) build_schedule<MODE>(sched, args);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = sched.prefix[kE] * (MODE == kWG && C8 ? 3 : 1);

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      uint32_t it = 0;
      bool ok = true;
      const uint64_t keep = policy_evict_last();
      for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
        const Tile t = decode_tile<MODE, C8>(sched, args, L);
        const CUtensorMap *mA = &tmA0, *mB = &tmB0;  // kWG
        if constexpr (MODE == kWG && C8 != 0) {
          if (t.part) {
            mA = &tmA1;
            mB = t.part == 1 ? &tmB1 : &more.b2;
          }
        }
        for (int kb = 0; kb < t.nkb; ++kb, ++it) {
          const int s = it % S;
          const uint32_t ph = (it / S) & 1u;
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], MODE == kDX ? A_BYTES + args.bn * BK * 2 : STAGE);
          uint8_t* a = sA + s * A_BYTES;
          uint8_t* b = sB + s * B_BYTES;
          if (MODE == kDH) {
            tma_load_2d_hint(a, &tmA0, &full[s], kb * BK, t.m0, keep);
#pragma unroll
            for (int c = 0; c < 4; ++c) tma_load_3d_hint(b + c * CHUNK, &tmB0, &full[s], kb * BK, t.n0 + 64 * c, t.e, keep);
          } else if (MODE == kDX) {
            const bool first = kb < args.half_kb;
            const int k0 = (first ? kb : kb - args.half_kb) * BK;
            tma_load_2d_hint(a, first ? &tmA0 : &tmA1, &full[s], k0, t.m0, keep);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (64 * c < args.bn)
                tma_load_3d_hint(b + c * CHUNK, first ? &tmB0 : &tmB1, &full[s], k0, t.n0 + 64 * c, t.e, keep);
          } else {
            const int r0 = t.row0 + kb * BK;
            tma_load_3d_hint(a, mA, &full[s], 0, r0, t.m0 / 64, keep);
            tma_load_3d_hint(b, mB, &full[s], 0, r0, t.n0 / 64, keep);
            *issued_kb = it + 1;
          }
        }
      }
      if (!ok) {
        flag_error(args.err, MOE_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      const uint32_t first = it > (uint32_t)S ? it - S : 0u;
      for (uint32_t j = first; j < it; ++j) mbar_wait(&full[j % S], (j / S) & 1u, nullptr, 100000000ull);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    // Lane 0 alone waits and issues, as in the forward GEMMs: a warp-wide loop
    // with a shuffle and a warp sync per K block held the dH and dx kernels
    // 25-35% below the MMA rate.
    if (lane == 0) {
      constexpr bool kMN = MODE == kWG;
      const int bn = MODE == kDX ? args.bn : BN;
      const uint32_t IDESC = idesc_bf16_f32(BM, bn, kMN, kMN);
      const uint32_t IDESC_M64 = idesc_bf16_f32(64, bn, kMN, kMN);
      uint32_t it = 0, tc = 0, zphase = 0;  // zphase: parity bit per stage of `zeroed`
      bool ok = true, issued = false;
      for (int L = blockIdx.x; L < total && ok; L += gridDim.x, ++tc) {
        const Tile t = decode_tile<MODE, C8>(sched, args, L);
        // a row block of at most 64 rows (an expert's last) runs M = 64 MMAs
        const uint32_t idesc = (MODE != kWG && t.rows <= 64) ? IDESC_M64 : IDESC;
        const uint32_t buf = tc & 1u;
        const uint32_t tph = (tc >> 1) & 1u;
        if (!mbar_wait(&tempty[buf], tph ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * kAccStride;
        for (int kb = 0; kb < t.nkb; ++kb, ++it) {
          const int s = it % S;
          const uint32_t ph = (it / S) & 1u;
          // K steps of 16 rows issued for this block: the expert's last block
          // issues only the steps that hold its rows; when the last such step
          // also holds rows past the expert's end, the zeroing warp clears them
          // in both operands and releases the stage on zeroed[s] instead.
          int ksteps = BK / 16;
          bool ragged = false;
          if (MODE == kWG) {
            const int valid = t.nrows - kb * BK;
            if (valid < BK) {
              ksteps = (valid + 15) / 16;
              ragged = ksteps * 16 > valid;
            }
          }
          if (ragged) {
            if (!mbar_wait(&zeroed[s], (zphase >> s) & 1u, abort_flag)) {
              ok = false;
              break;
            }
            zphase ^= 1u << s;
          } else if (!mbar_wait(&full[s], ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + s * A_BYTES);
          const uint32_t b_addr = smem_u32(sB + s * B_BYTES);
          auto mma_step = [&](int kk) {
            uint64_t ad, bd;
            if (kMN) {
              ad = sw128_desc(a_addr + kk * 2048, CHUNK, 1024);
              bd = sw128_desc(b_addr + kk * 2048, CHUNK, 1024);
            } else {
              ad = sw128_desc(a_addr + kk * 32, 16, 1024);
              bd = sw128_desc(b_addr + kk * 32, 16, 1024);
            }
            umma_bf16(d_tmem, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
          };
          // full K blocks issue their four steps without a branch: a bound check
          // inside this loop cost the weight gradients 11% of the MMA rate
          if (ksteps == BK / 16) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) mma_step(kk);
          } else {
            for (int kk = 0; kk < ksteps; ++kk) mma_step(kk);
          }
          issued = true;
          umma_commit(&empty[s]);
        }
        if (!ok) break;
        umma_commit(&tfull[buf]);
      }
      if (!ok) {
        flag_error(args.err, MOE_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (issued) {
        umma_commit(drain);
        mbar_wait(drain, 0, nullptr, 100000000ull);
      }
    }
  } else if (warp == Warps<MODE, C8>::kZeroWarp) {
    // ------------------------------------------------ ragged-row zeroing (kWG)
    // The tile's last K block may hold rows past the expert's end (the next
    // expert's rows, or rows past the kept ones): once the stage has landed,
    // zero those rows of the last 16-row step in all six 8 KB chunks (a row is
    // 128 bytes of a chunk, so the swizzle does not matter), make the writes
    // visible to the tensor core and release the stage to the MMA warp.  Every
    // lane waits for the stage itself, so its stores follow the TMA's.
    uint32_t it = 0;
    for (int L = blockIdx.x; L < total; L += gridDim.x) {
      const Tile t = decode_tile<MODE, C8>(sched, args, L);
      const uint32_t it_last = it + (uint32_t)t.nkb - 1u;
      it += (uint32_t)t.nkb;
      if (t.nkb == 0) continue;
      const int valid = t.nrows - (t.nkb - 1) * BK;
      const int pad = (valid + 15) / 16 * 16 - valid;
      if (valid >= BK || pad == 0) continue;
      const int s = it_last % S;
      // bounded: the producer issues this K block's loads unless the kernel aborts
      const uint64_t t0 = globaltimer_ns();
      bool go = true;
      while ((int)(*issued_kb - it_last) <= 0) {
        if (*abort_flag || globaltimer_ns() - t0 > 2000000000ull) {
          go = false;
          break;
        }
        __nanosleep(32);
      }
      if (!go || !mbar_wait(&full[s], (it_last / S) & 1u, abort_flag)) {
        if (!*abort_flag) {
          if (lane == 0) flag_error(args.err, MOE_DEVERR_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
      const int per_chunk = pad * 8;  // 16-byte pieces
      for (int i = lane; i < 6 * per_chunk; i += 32) {
        const int c = i / per_chunk;
        const int j = i - c * per_chunk;
        uint8_t* chunk = c < 2 ? sA + s * A_BYTES + c * CHUNK : sB + s * B_BYTES + (c - 2) * CHUNK;
        *reinterpret_cast<uint4*>(chunk + valid * 128 + j * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&zeroed[s]);
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;
    // column chunks of 32 this warp covers: all 8, or one half with 8 epilogue warps
    constexpr int kSplit = Warps<MODE, C8>::kEpi / 4;
    const int half = kSplit == 1 ? 0 : (warp - 2) / 4;
    const int c_begin = half * (BN / 32) / kSplit, c_end = c_begin + (BN / 32) / kSplit;
    uint32_t tc = 0;
    for (int L = blockIdx.x; L < total; L += gridDim.x, ++tc) {
      const Tile t = decode_tile<MODE, C8>(sched, args, L);
      const uint32_t buf = tc & 1u;
      const uint32_t tph = (tc >> 1) & 1u;
      // tile row of this thread; M = 64 accumulators hold row 16 q + i in lane i (< 16) of quarter q
      const int r = (MODE != kWG && t.rows <= 64) ? (lane < 16 ? q * 16 + lane : BM) : q * 32 + lane;
      // kDH, C8: codes of a 32-column chunk, 2 x 16 bytes of G and of U.  The
      // first chunk's and the scales do not wait for the products; the next
      // chunk's are loaded while one is computed.
      constexpr int NC = BN / 32 / kSplit;  // chunks of this warp
      const bool valid = r < t.rows;
      const int64_t row = t.m0 + r;
      const int64_t base = row * args.ld + t.n0 + c_begin * 32;
      float w = 0.f;
      uint4 qg[2], qu[2];
      uint2 sg4[NC / 4] = {}, su4[NC / 4] = {};  // four bf16 scales each
      // a checkpoint is 16-byte aligned, and its parts lie multiples of 256 bytes apart
      const bool sectors = (reinterpret_cast<uintptr_t>(args.codes.g) & 31u) == 0;
      auto load_chunk = [&](int c, uint4 (&a)[2], uint4 (&b)[2]) {
        const uint4* g = reinterpret_cast<const uint4*>(args.codes.g + base + c * 32);
        const uint4* u = reinterpret_cast<const uint4*>(args.codes.u + base + c * 32);
        if (sectors) {
          load32_once(g, a);
          load32_once(u, b);
        } else {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            a[p] = __ldg(g + p);
            b[p] = __ldg(u + p);
          }
        }
      };
      if (MODE == kDH && C8 && valid) {
        w = __ldg(args.row_scale + row);
#pragma unroll
        for (int i = 0; i < NC / 4; ++i) {
          sg4[i] = __ldg(reinterpret_cast<const uint2*>(args.codes.sg + base / 32) + i);
          su4[i] = __ldg(reinterpret_cast<const uint2*>(args.codes.su + base / 32) + i);
        }
        load_chunk(0, qg, qu);
      }
      if (!mbar_wait(&tfull[buf], tph, abort_flag)) {
        if (lane == 0) flag_error(args.err, MOE_DEVERR_TIMEOUT);
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t tacc = tmem_base + buf * kAccStride + ((uint32_t)(q * 32) << 16);
      if (MODE == kDH && C8) {
        const uint32_t tmine = tacc + c_begin * 32;
        const f32x2 w2 = pack2(w, w), one = pack2(1.f, 1.f), minus1 = pack2(-1.f, -1.f);
        f32x2 dot = pack2(0.f, 0.f);
        // The three results go out 32 rows x 32 columns at a time by TMA from shared
        // memory (rows of 64 bytes, 64-byte swizzle), two buffers a warp: stored by
        // the threads, each 16 bytes of its own row, they kept the load/store unit at
        // 32 lines an instruction and the tile at 38K clocks.  A warp whose rows pass
        // the expert's end stores its valid rows itself.
        const bool whole = (q + 1) * 32 <= t.rows && t.rows > 64;
        uint8_t* stage0 = sOut + (warp - 2) * (OUT_BYTES / Warps<MODE, C8>::kEpi);
        int turn = 0;
        auto put = [&](const CUtensorMap* map, const uint4 (&v)[4], int x) {
          uint8_t* st = stage0 + (turn & 1) * 2048;
          ++turn;
          if (lane == 0) bulk_wait_group_read<1>();  // the store that last read this buffer is done with it
          __syncwarp();
          uint4* line = reinterpret_cast<uint4*>(st + lane * 64);
#pragma unroll
          for (int j = 0; j < 4; ++j) line[j ^ ((lane >> 1) & 3)] = v[j];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(map, st, x, t.m0 + q * 32);
            bulk_commit_group();
          }
        };
        // (one chunk's code: unrolled over the chunks, the warps waited for
        // instructions a quarter of the time)
#pragma unroll 1
        for (int c = 0; c < NC; ++c) {
          uint32_t v[32];
          tmem_ld32(tmine + c * 32, v);
          const bool more = c + 1 < NC;
          uint4 ng[2], nu[2];
          if (valid && more) load_chunk(c + 1, ng, nu);
          tmem_wait_ld();
          uint4 kg[4], ku[4], kh[4];
          if (valid) {
            const uint2 pg = NC == 8 && c >= 4 ? sg4[NC / 4 - 1] : sg4[0], pu = NC == 8 && c >= 4 ? su4[NC / 4 - 1] : su4[0];
            const uint32_t wg = (c & 2) ? pg.y : pg.x, wu = (c & 2) ? pu.y : pu.x;
            const float sg = __uint_as_float((c & 1) ? wg & 0xffff0000u : wg << 16);
            const float su = __uint_as_float((c & 1) ? wu & 0xffff0000u : wu << 16);
            const f32x2 sg2 = pack2(sg, sg), su2 = pack2(su, su);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              uint32_t og[4], ou[4], oh[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // two values at a time
                const int word = 2 * p + (i >> 1);
                const f32x2 g = mul2(sg2, codes2((&qg[word >> 2].x)[word & 3], i & 1));
                const f32x2 u = mul2(su2, codes2((&qu[word >> 2].x)[word & 3], i & 1));
                const f32x2 dhu = pack2(__uint_as_float(v[p * 8 + 2 * i]), __uint_as_float(v[p * 8 + 2 * i + 1]));
                // the approximate quotient (2 ulp; 0 where e^-g passes 2^126, its
                // limit): the IEEE one held this epilogue at 65 us a tile
                float g0, g1;
                unpack2(g, g0, g1);
                const f32x2 sig = pack2(__fdividef(1.0f, 1.0f + __expf(-g0)), __fdividef(1.0f, 1.0f + __expf(-g1)));
                const f32x2 sl = mul2(g, sig);
                const f32x2 h = mul2(sl, u);
                dot = fma2(dhu, h, dot);
                const f32x2 dh = mul2(w2, dhu);
                // silu'(g) = sig + sl (1 - sig)
                og[i] = pack_bf16x2(mul2(mul2(dh, u), fma2(sl, fma2(sig, minus1, one), sig)));
                ou[i] = pack_bf16x2(mul2(dh, sl));
                oh[i] = pack_bf16x2(mul2(w2, h));
              }
              kg[p] = make_uint4(og[0], og[1], og[2], og[3]);
              ku[p] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
              kh[p] = make_uint4(oh[0], oh[1], oh[2], oh[3]);
            }
          }
          const int x = t.n0 + (c_begin + c) * 32;
          if (whole) {
            put(&tmA1, kg, x);
            put(&tmB1, ku, x);
            put(&tmOut, kh, x);
          } else if (valid) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const int64_t o = base + c * 32 + p * 8;
              __stcs(reinterpret_cast<uint4*>(args.dG + o), kg[p]);
              __stcs(reinterpret_cast<uint4*>(args.dU + o), ku[p]);
              __stcs(reinterpret_cast<uint4*>(args.hw + o), kh[p]);
            }
          }
          if (more) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              qg[p] = ng[p];
              qu[p] = nu[p];
            }
          }
        }
        if (valid) {
          float d0, d1;
          unpack2(dot, d0, d1);
          args.dw_part[(row * (int64_t)args.n_tiles + t.nb) * kSplit + half] = d0 + d1;
        }
      } else if (MODE == kDH) {
        const bool valid = r < t.rows;
        const int64_t row = t.m0 + r;
        const float w = valid ? __ldg(args.row_scale + row) : 0.f;
        const int64_t base = row * args.ld + t.n0;
        float dot = 0.f;
        // G, U, H of a 32-column chunk: 4 x 16 bytes each; the next chunk's are
        // loaded while this one is computed, so the loads overlap the math.  They
        // and the dG, dU stores stream through L2 (evict-first): each is touched
        // once here, and keeping them from pushing out the operand tiles made
        // the kernel 5% faster at Grok size
        uint4 qg[4], qu[4], qh[4];
        auto load_chunk = [&](int c, uint4 (&a)[4], uint4 (&b)[4], uint4 (&hh)[4]) {
          const int64_t o = base + c * 32;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            a[p] = __ldcs(reinterpret_cast<const uint4*>(args.G + o + p * 8));
            b[p] = __ldcs(reinterpret_cast<const uint4*>(args.U + o + p * 8));
            hh[p] = __ldcs(reinterpret_cast<const uint4*>(args.H + o + p * 8));
          }
        };
        if (valid) load_chunk(c_begin, qg, qu, qh);
#pragma unroll 1
        for (int c = c_begin; c < c_end; ++c) {
          uint32_t v[32];
          tmem_ld32(tacc + c * 32, v);
          const bool more = c + 1 < c_end;
          uint4 ng[4], nu[4], nh[4];
          if (valid && more) load_chunk(c + 1, ng, nu, nh);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const int64_t o = base + c * 32 + p * 8;
              float g[8], u[8], h[8];
              unpack8_bf16(qg[p], g);
              unpack8_bf16(qu[p], u);
              unpack8_bf16(qh[p], h);
              uint32_t og[4], ou[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float dg2[2], du2[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int j = 2 * i + k;
                  const float dhu = __uint_as_float(v[p * 8 + j]);
                  dot = fmaf(dhu, h[j], dot);
                  const float dh = w * dhu;
                  const float sg = 1.0f / (1.0f + __expf(-g[j]));
                  const float sl = g[j] * sg;
                  dg2[k] = dh * u[j] * (sg * (1.0f + g[j] * (1.0f - sg)));
                  du2[k] = dh * sl;
                }
                og[i] = pack_bf16x2(dg2[0], dg2[1]);
                ou[i] = pack_bf16x2(du2[0], du2[1]);
              }
              __stcs(reinterpret_cast<uint4*>(args.dG + o), make_uint4(og[0], og[1], og[2], og[3]));
              __stcs(reinterpret_cast<uint4*>(args.dU + o), make_uint4(ou[0], ou[1], ou[2], ou[3]));
            }
          }
          if (more) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              qg[p] = ng[p];
              qu[p] = nu[p];
              qh[p] = nh[p];
            }
          }
        }
        if (valid) args.dw_part[row * (int64_t)args.n_tiles * kSplit + t.nb * kSplit + half] = dot;
      } else if (MODE == kDX) {
        int tok = -1;
        if (r < t.rows) {
          tok = __ldg(args.perm + t.m0 + r);
          if (tok < 0 || (int64_t)tok >= args.n_tok) {
            flag_error(args.err, MOE_DEVERR_SLOT_INDEX);
            tok = -1;
          }
        }
        float* dst = args.out + (int64_t)(tok < 0 ? 0 : tok) * args.ld + t.n0;
#pragma unroll 1
        for (int c = 0; c < args.bn / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(tacc + c * 32, v);
          tmem_wait_ld();
          if (tok >= 0) {
            float4* d4 = reinterpret_cast<float4*>(dst + c * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              atomicAdd(d4 + i, make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                            __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])));
          }
        }
      } else if constexpr (C8 != 0 && MODE == kWG) {
        // as below with 32 rows x 64 bf16 columns (128 bytes) per store
        const CUtensorMap* mOut = t.part == 0 ? &tmOut : (t.part == 1 ? &more.out1 : &more.out2);
        const bool zero = t.nkb == 0;
        uint8_t* stage0 = sOut + (q * 2) * OUT_STAGE;
        const int y = t.e * args.wg[t.part].M + t.m0 + q * 32;
#pragma unroll 1
        for (int c = 0; c < BN / 64; ++c) {
          uint32_t v[32], v2[32];
          tmem_ld32(tacc + c * 64, v);
          tmem_ld32(tacc + c * 64 + 32, v2);
          tmem_wait_ld();
          uint8_t* st = stage0 + (c & 1) * OUT_STAGE;
          if (lane == 0) bulk_wait_group_read<1>();
          __syncwarp();
          uint4* row = reinterpret_cast<uint4*>(st + lane * 128);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t* s8 = j < 4 ? v + 8 * j : v2 + 8 * (j - 4);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[i] = zero ? 0u : pack_bf16x2(__uint_as_float(s8[2 * i]), __uint_as_float(s8[2 * i + 1]));
            row[j ^ (lane & 7)] = make_uint4(o[0], o[1], o[2], o[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(mOut, st, t.n0 + c * 64, y);
            bulk_commit_group();
          }
        }
      } else {
        // 32 rows x 32 columns per TMA store: lane = row, its 8 16-byte pieces
        // placed with the 128-byte swizzle (piece j of row r at j ^ (r % 8))
        const bool zero = t.nkb == 0;
        uint8_t* stage0 = sOut + (q * 2) * OUT_STAGE;
        const int y = t.e * args.wg[t.part].M + t.m0 + q * 32;
#pragma unroll 1
        for (int c = 0; c < BN / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(tacc + c * 32, v);
          tmem_wait_ld();
          uint8_t* st = stage0 + (c & 1) * OUT_STAGE;
          if (lane == 0) bulk_wait_group_read<1>();  // the store that last read this buffer is done with it
          __syncwarp();
          float4* row = reinterpret_cast<float4*>(st + lane * 128);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            row[j ^ (lane & 7)] = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                                       : make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                                     __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmOut, st, t.n0 + c * 32, y);
            bulk_commit_group();
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&tempty[buf]);
    }
  }

  // tile stores still in flight must finish before the CTA (and its shared memory) goes
  if ((MODE == kWG || (MODE == kDH && C8)) && warp >= 2 && lane == 0) bulk_wait_group_all();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <int MODE, int C8 = 0>
cudaError_t launch_bwd(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0, const CUtensorMap& b1,
                       const CUtensorMap& out, const BwdArgs& args, cudaStream_t s, const Ctx& ctx,
                       const MoreMaps<MODE, C8>& more = {}) {
  auto kern = bwd_gemm_kernel<MODE, C8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(ctx.num_sms), dim3(Warps<MODE, C8>::kThreads), SMEM_BYTES, s, no_extra_attr(), a0, a1, b0,
                 b1, out, more, args);
  return e != cudaSuccess ? e : cudaGetLastError();
}

BwdArgs base_args(const moe_config_t& c, const int32_t* offsets, const Ctx& ctx) {
  BwdArgs a = {};
  a.offsets = offsets;
  a.rows_alloc = slot_rows(c);
  a.n_tok = c.T;
  a.err = ctx.err;
  return a;
}

bool map_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, uint32_t box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t str[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {64, box_rows};
  return encode_tmap(m, base, 2, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// [rows, cols] bf16 results stored 32 x 32 at a time, rows of 64 bytes in shared memory
bool map_out(CUtensorMap* m, const void* base, int64_t rows, int64_t cols) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t str[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {32, 32};
  return encode_tmap(m, base, 2, dims, str, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

// [E, R, C] weights, box of 64 columns x 64 rows of one expert
bool map_weights(CUtensorMap* m, const void* base, int E, int64_t R, int64_t C) {
  const uint64_t dims[3] = {(uint64_t)C, (uint64_t)R, (uint64_t)E};
  const uint64_t str[2] = {(uint64_t)C * 2, (uint64_t)R * C * 2};
  const uint32_t box[3] = {64, 64, 1};
  return encode_tmap(m, base, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

int bwd_dh_parts_per_tile() { return Warps<kDH>::kEpi / 4; }
int bwd_dh_c8_parts_per_tile(const moe_config_t& c) { return c.d < 2048 ? 2 : 1; }

cudaError_t launch_bwd_dh(const moe_config_t& c, const void* dout_perm, const int32_t* offsets, const void* wd,
                          const void* G, const void* U, const void* H, const float* row_scale, void* dG, void* dU,
                          float* dw_part, cudaStream_t s, const Ctx& ctx) {
  const int64_t rows = slot_rows(c);
  if (rows == 0) return cudaSuccess;
  CUtensorMap ta, tb;
  // W_down [E, f, d] read K-major: rows = f (N), columns = d (K)
  if (!map_rows(&ta, dout_perm, rows, c.d, 128) || !map_weights(&tb, wd, c.E, c.f, c.d))
    return cudaErrorInvalidValue;
  BwdArgs a = base_args(c, offsets, ctx);
  a.n_tiles = (int)(c.f / BN);
  a.num_kb = (int)(c.d / BK);
  a.row_scale = row_scale;
  a.G = static_cast<const __nv_bfloat16*>(G);
  a.U = static_cast<const __nv_bfloat16*>(U);
  a.H = static_cast<const __nv_bfloat16*>(H);
  a.dG = static_cast<__nv_bfloat16*>(dG);
  a.dU = static_cast<__nv_bfloat16*>(dU);
  a.dw_part = dw_part;
  a.ld = c.f;
  return launch_bwd<kDH>(ta, ta, tb, tb, ta, a, s, ctx);
}

cudaError_t launch_bwd_dh_c8(const moe_config_t& c, const void* dout_perm, const int32_t* offsets, const void* wd,
                             const Codes8& codes, const float* row_scale, void* dG, void* dU, void* hw, float* dw_part,
                             cudaStream_t s, const Ctx& ctx) {
  const int64_t rows = slot_rows(c);
  if (rows == 0) return cudaSuccess;
  CUtensorMap ta, tb, tg, tu, th;
  if (!map_rows(&ta, dout_perm, rows, c.d, 128) || !map_weights(&tb, wd, c.E, c.f, c.d) || !map_out(&tg, dG, rows, c.f) ||
      !map_out(&tu, dU, rows, c.f) || !map_out(&th, hw, rows, c.f))
    return cudaErrorInvalidValue;
  BwdArgs a = base_args(c, offsets, ctx);
  a.n_tiles = (int)(c.f / BN);
  a.num_kb = (int)(c.d / BK);
  a.row_scale = row_scale;
  a.codes = codes;
  a.hw = static_cast<__nv_bfloat16*>(hw);
  a.dG = static_cast<__nv_bfloat16*>(dG);
  a.dU = static_cast<__nv_bfloat16*>(dU);
  a.dw_part = dw_part;
  a.ld = c.f;
  if (bwd_dh_c8_parts_per_tile(c) == 2) return launch_bwd<kDH, 8>(ta, tg, tb, tu, th, a, s, ctx);
  return launch_bwd<kDH, 4>(ta, tg, tb, tu, th, a, s, ctx);
}

cudaError_t launch_bwd_dx(const moe_config_t& c, const void* dG, const void* dU, const int32_t* offsets,
                          const void* wg, const void* wu, const int32_t* perm, float* dx32, cudaStream_t s,
                          const Ctx& ctx) {
  const int64_t rows = slot_rows(c);
  if (rows == 0) return cudaSuccess;
  CUtensorMap ta0, ta1, tb0, tb1;
  // W_gate / W_up [E, d, f] read K-major: rows = d (N), columns = f (K)
  if (!map_rows(&ta0, dG, rows, c.f, 128) || !map_rows(&ta1, dU, rows, c.f, 128) ||
      !map_weights(&tb0, wg, c.E, c.d, c.f) || !map_weights(&tb1, wu, c.E, c.d, c.f))
    return cudaErrorInvalidValue;
  BwdArgs a = base_args(c, offsets, ctx);
  a.bn = tile_columns(c, c.d, {256, 192}, ctx.num_sms);
  a.n_tiles = (int)(c.d / a.bn);
  a.half_kb = (int)(c.f / BK);
  a.num_kb = 2 * a.half_kb;
  a.perm = perm;
  a.out = dx32;
  a.ld = c.d;
  return launch_bwd<kDX>(ta0, ta1, tb0, tb1, ta0, a, s, ctx);
}

namespace {

// Rows [rows, C] viewed as [C / 64 chunks][rows][64]: one box = `chunks` chunks of 64 x 64.
bool map_chunks(CUtensorMap* m, const void* base, int64_t rows, int64_t C, uint32_t chunks) {
  const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)(C / 64)};
  const uint64_t str[2] = {(uint64_t)C * 2, 128};
  const uint32_t box[3] = {64, 64, chunks};
  return encode_tmap(m, base, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// dW [E * M, N] stored 32 rows x 128 bytes at a time from the swizzled staging tiles
bool map_dw(CUtensorMap* m, const void* dW, int64_t rows, int64_t N, bool bf16) {
  const uint32_t esz = bf16 ? 2 : 4;
  const uint64_t dims[2] = {(uint64_t)N, (uint64_t)rows};
  const uint64_t str[1] = {(uint64_t)N * esz};
  const uint32_t box[2] = {128 / esz, 32};
  return encode_tmap_dtype(m, dW, 2, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B,
                           bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32);
}

WgShape wg_shape(int64_t M, int64_t N, bool m_outer) {
  return {(int)M, (int)(M / BM), (int)(N / BN), m_outer ? 1 : 0};
}

}  // namespace

cudaError_t launch_bwd_wgrad(const moe_config_t& c, const void* a_rows, int64_t M, const void* b_rows, int64_t N,
                             const int32_t* offsets, float* dW, bool m_outer, cudaStream_t s, const Ctx& ctx) {
  const int64_t rows = slot_rows(c);
  if (rows == 0 || M % BM != 0 || N % BN != 0) return rows == 0 ? cudaSuccess : cudaErrorInvalidValue;
  CUtensorMap ta, tb, to;
  if (!map_chunks(&ta, a_rows, rows, M, 2) || !map_chunks(&tb, b_rows, rows, N, 4) || !map_dw(&to, dW, c.E * M, N, false))
    return cudaErrorInvalidValue;
  BwdArgs a = base_args(c, offsets, ctx);
  a.wg[0] = wg_shape(M, N, m_outer);
  a.out = dW;
  return launch_bwd<kWG>(ta, ta, tb, tb, to, a, s, ctx);
}

cudaError_t launch_bwd_wgrads_c8(const moe_config_t& c, const void* hw, const void* dout_perm, const void* x_perm,
                                 const void* dG, const void* dU, const int32_t* offsets, void* dw_down, void* dw_gate,
                                 void* dw_up, cudaStream_t s, const Ctx& ctx) {
  const int64_t rows = slot_rows(c);
  if (rows == 0 || c.d % BN != 0 || c.f % BN != 0) return rows == 0 ? cudaSuccess : cudaErrorInvalidValue;
  CUtensorMap ta0, ta1, tb0, tb1, to;
  WgMaps more;
  if (!map_chunks(&ta0, hw, rows, c.f, 2) || !map_chunks(&tb0, dout_perm, rows, c.d, 4) ||
      !map_dw(&to, dw_down, c.E * c.f, c.d, true) || !map_chunks(&ta1, x_perm, rows, c.d, 2) ||
      !map_chunks(&tb1, dG, rows, c.f, 4) || !map_chunks(&more.b2, dU, rows, c.f, 4) ||
      !map_dw(&more.out1, dw_gate, c.E * c.d, c.f, true) || !map_dw(&more.out2, dw_up, c.E * c.d, c.f, true))
    return cudaErrorInvalidValue;
  BwdArgs a = base_args(c, offsets, ctx);
  a.wg[0] = wg_shape(c.f, c.d, c.f >= c.d);
  a.wg[1] = a.wg[2] = wg_shape(c.d, c.f, c.d >= c.f);
  return launch_bwd<kWG, 4>(ta0, ta1, tb0, tb1, to, a, s, ctx, more);
}

}  // namespace moe
