// Expert GEMMs on microscaled 4-bit weights and 8-bit activations, on the
// block-scaled tcgen05 MMA (kind::mxf8f6f4: e4m3 rows x e2m1 weights, one e8m0
// scale for 32 values along K on both sides, fp32 accumulation).
//
//   gate/up : H[r, n] = silu(sum_k x^ g^) * (sum_k x^ u^), 128 gate and the 128
//             matching up columns of a tile in one 128 x 256 accumulator; the
//             epilogue holds 32 consecutive columns of a row per thread, one
//             block of the next GEMM's K, so it writes H as e4m3 codes and
//             scales without an exchange between threads.
//   down    : Y[r, n] = row_scale[r] * sum_k h^ d^, 256 columns; added into the
//             tokens' fp32 sums (two terms a token: the order does not matter),
//             or stored as K-split partials where there are few rows.
// Few rows (decode): the weights on the MMA's other side, see Ring.
//
// The weights stay 4 bits until the tensor core: TMA reads packed codes and
// spreads 16 of them over 16 bytes of shared memory (8 bytes of padding), the
// form in which the MMA takes 4-bit operands beside 8-bit ones, so no thread
// decodes anything.  Memory traffic is 0.53 bytes a weight, which bounds calls
// of few rows; the MMA runs at twice the bf16 rate, which bounds the others.
//
// TMEM: two 128 x 256 fp32 accumulators would fill all 512 columns and leave
// none for the scales, so the second starts 48 columns early, [208, 464), and
// the scales live in [464, 512): one set a stage, 4 columns for the rows and 8
// for the weights.  The epilogue reads the 48 shared columns first and releases
// them; the next tile's MMAs start then, while the rest is still being read.
//
// Row tiles of 128 (or 32 or 64, see Ring); a tile with at most 96 rows loads its rows
// in boxes of 32, so that a decode tile moves 4 KB of rows beside 17 KB of
// weights a stage.
// Rows past an expert's end are computed from whatever is there and never
// stored (rows of an MMA are independent).  Schedule, roles and bounded waits as
// in the bf16 GEMMs (ffn_tc.cu): persistent CTAs, warp 0 TMA, warp 1 MMA, warps
// 2-5 epilogue, and warps 6-9 for the scales.
#include <cuda.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kE = 8;
constexpr int BK = 128;
constexpr int kThreads = 320;          // 10 warps: TMA, MMA, 4 epilogue, 4 scales
constexpr int B_HALF = 128 * BK;       // 16 KB: 128 channels x 128 codes, spread
constexpr int B_BYTES = 2 * B_HALF;
constexpr int B_TX = B_BYTES / 2;      // bytes that the spreading loads report: those read, not the padding
constexpr int kTmemCols = 512;
constexpr int kAccSecond = 208;        // first column of the second accumulator
constexpr int kScaleCol = 464;         // kScaleSets sets of 12 columns
constexpr int kScaleSets = 4;
static_assert(kScaleCol + 12 * kScaleSets <= kTmemCols, "TMEM columns");
constexpr int kGroupSlots = 3;         // groups of scales in shared memory

// BM rows a tile: 128, or 32 or 64 where few rows an expert are expected.  The
// block-scaled MMA takes 128 rows on its A side at least, so these put the
// weights there (two MMAs of 128 channels x BM rows for 256 channels) and the rows
// on the B side: an MMA then costs its 4 KB of weights, and the accumulators are
// 2 BM columns, lane = channel, column = row.  With the rows on the A side, padded
// to 128, the tensor core was busy for 60% of the time and gate/up of Grok-1
// decode (T 32) took 307 us, where it takes 257 so (1.71 GB of weights and scales:
// 6.67 TB/s).  The room of the rows goes to a fifth stage (4: 5 to 6% slower at 64
// rows) and to scales further ahead: they come from DRAM here, and with 4 K blocks
// ahead the MMAs waited for them (338 us).
template <int BM>
struct Ring {
  static constexpr bool kSwap = BM < 128;           // weights on the A side
  static constexpr int kStages = kSwap ? 5 : 4;
  static constexpr int A_BYTES = BM * BK;
  static constexpr int kGroup = BM == 32 ? 8 : (BM == 64 ? 5 : 4);  // K blocks whose scales are loaded together
  static constexpr int GROUP_BYTES = 3 * kGroup * 512;
  static constexpr int kBars = 2 * kStages + 2 + 2 + kScaleSets + 2 * kGroupSlots + 1;
  static constexpr int SMEM_BYTES = 1024 + kStages * (A_BYTES + B_BYTES) + kGroupSlots * GROUP_BYTES + kBars * 8 + 16;
  static_assert(SMEM_BYTES + 256 <= 227 * 1024, "shared memory budget");
};

enum Mode { kGateUp = 0, kDownSum = 1, kDownParts = 2 };

struct MxArgs {
  const int32_t* offsets;    // [E + 1]
  int64_t rows_alloc;
  int n_tiles;               // gate/up: f / 128;  down: d / bn
  int bn;                    // columns of a tile: gate/up 128 (and 128 up), down 256, 192 or 128
  int num_kb;                // K / 128
  int splits;                // K splits (kDownParts; 1 otherwise)
  const uint8_t* a_scales;   // [row tiles][K / 128][512]
  const uint8_t* b_scales0;  // [E][N / 128][K / 128][512]
  const uint8_t* b_scales1;  // gate/up: of the up weights
  int nb_scales;             // N / 128
  uint8_t* h;                // gate/up: codes [rows, f]
  uint8_t* h_scales;         // gate/up: [row tiles][f / 128][512]
  float* out;                // down: sums [T, d] or partials [splits][rows][d]
  int64_t ld;                // gate/up: f;  down: d
  const float* row_scale;    // down; NULL means 1
  const int32_t* perm;       // kDownSum
  int64_t n_tok;
  int* err;
};

struct Sched {
  int offs[kE + 1];
  int mt[kE];
  int tile0[kE];             // first row tile of the expert's scales
  int prefix[kE + 1];
};

struct Tile {
  int e, m0, rows, nt, kb0, kb1, split;
  int mtile, in_mtile;  // 128-row tile of the rows' scales, and the first row's place in it
};

template <int BM>
__device__ __forceinline__ Tile decode_tile(const Sched& s, const MxArgs& a, int L) {
  int e = 0;
#pragma unroll
  for (int k = 1; k < kE; ++k)
    if (L >= s.prefix[k]) e = k;
  int local = L - s.prefix[e];
  Tile t;
  t.e = e;
  t.split = 0;
  if (a.splits > 1) {
    t.split = local % a.splits;
    local /= a.splits;
  }
  t.nt = local / s.mt[e];
  const int mi = local - t.nt * s.mt[e];
  t.m0 = s.offs[e] + mi * BM;
  t.mtile = s.tile0[e] + mi * BM / 128;
  t.in_mtile = mi * BM % 128;
  const int left = s.offs[e + 1] - t.m0;
  t.rows = left < BM ? left : BM;
  t.kb0 = a.num_kb * t.split / a.splits;
  t.kb1 = a.num_kb * (t.split + 1) / a.splits;
  return t;
}

template <int BM>
__device__ __forceinline__ void build_schedule(Sched& sched, const MxArgs& args) {
  bool ok = true;
  int prev = 0;
  for (int k = 0; k <= kE; ++k) {
    const int v = args.offsets[k];
    sched.offs[k] = v;
    if (v < prev || (int64_t)v > args.rows_alloc) ok = false;
    prev = v;
  }
  int acc = 0, tiles = 0;
  for (int k = 0; k < kE; ++k) {
    const int n = ok ? sched.offs[k + 1] - sched.offs[k] : 0;
    sched.mt[k] = (n + BM - 1) / BM;
    sched.tile0[k] = tiles;
    sched.prefix[k] = acc;
    tiles += (n + 127) / 128;
    acc += sched.mt[k] * args.n_tiles * args.splits;
  }
  sched.prefix[kE] = acc;
  if (!ok) flag_error(args.err, MOE_DEVERR_OFFSETS);
}

template <int MODE, int BM>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                    const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                    const MxArgs args) {
  using R = Ring<BM>;
  constexpr int S = R::kStages;
  // columns of a tile (a variable only where the width is chosen)
  const int bn = MODE == kGateUp ? 128 : (MODE == kDownParts ? 256 : args.bn);
  constexpr int kGroup = R::kGroup, GROUP_BYTES = R::GROUP_BYTES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * R::A_BYTES;
  uint8_t* sG = sB + S * B_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sG + kGroupSlots * GROUP_BYTES);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;        // accumulator 0 / 1 complete
  uint64_t* tshared = tfull + 2;      // [0]: the columns both accumulators use have been read
                                      // (swapped: accumulator 0 / 1 has been read)
  uint64_t* sfull = tshared + 2;      // scale set written
  uint64_t* gfull = sfull + kScaleSets;  // group of scales landed
  uint64_t* gfree = gfull + kGroupSlots; // ... and read
  uint64_t* drain = gfree + kGroupSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ Sched sched;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&tfull[0], 1);
    mbar_init(&tfull[1], 1);
    mbar_init(&tshared[0], 128);
    mbar_init(&tshared[1], 128);
    for (int s = 0; s < kScaleSets; ++s) mbar_init(&sfull[s], 4);
    for (int s = 0; s < kGroupSlots; ++s) {
      mbar_init(&gfull[s], 1);
      mbar_init(&gfree[s], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 1) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmA32);
    prefetch_tmap(&tmB0);
    prefetch_tmap(&tmB1);
  }
  pdl_wait();
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  if (warp == 2 && lane == 0) build_schedule<BM>(sched, args);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = sched.prefix[kE];

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      uint32_t it = 0;
      bool ok = true;
      const uint64_t keep = policy_evict_last();
      for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
        const Tile t = decode_tile<BM>(sched, args, L);
        const int boxes = t.rows > 96 ? 0 : (t.rows + 31) / 32;
        // boxes of 128 channels; a tile of 192 columns takes three of 64 (64 for
        // all made the down pass 17 to 24% slower)
        const int box_n = bn % 128 == 0 ? 128 : 64;
        const uint32_t bytes = (boxes ? (uint32_t)boxes * 32 * BK : R::A_BYTES) +
                               (MODE == kGateUp ? B_TX : (uint32_t)bn * BK / 2);
        const int n0 = t.nt * bn;
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const int s = it % S;
          const uint32_t ph = (it / S) & 1u;
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], bytes);
          uint8_t* a = sA + s * R::A_BYTES;
          uint8_t* b = sB + s * B_BYTES;
          if (MODE == kGateUp) {
            tma_load_3d_hint(b, &tmB0, &full[s], kb * BK, n0, t.e, keep);
            tma_load_3d_hint(b + B_HALF, &tmB1, &full[s], kb * BK, n0, t.e, keep);
          } else {
            tma_load_3d_hint(b, &tmB0, &full[s], kb * BK, n0, t.e, keep);
            if (bn > box_n) tma_load_3d_hint(b + box_n * BK, &tmB0, &full[s], kb * BK, n0 + box_n, t.e, keep);
            if (bn > 2 * box_n) tma_load_3d_hint(b + 2 * box_n * BK, &tmB0, &full[s], kb * BK, n0 + 2 * box_n, t.e, keep);
          }
          if (boxes == 0) {
            tma_load_2d_hint(a, &tmA, &full[s], kb * BK, t.m0, keep);
          } else {
            for (int i = 0; i < boxes; ++i)
              tma_load_2d_hint(a + i * 32 * BK, &tmA32, &full[s], kb * BK, t.m0 + 32 * i, keep);
          }
        }
      }
      if (!ok) {
        flag_error(args.err, MOE_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
      // drain: every issued load must land before the CTA can exit
      const uint32_t first = it > (uint32_t)S ? it - S : 0u;
      for (uint32_t j = first; j < it; ++j) mbar_wait(&full[j % S], (j / S) & 1u, nullptr, 100000000ull);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    // The whole warp runs the loop and one elected lane issues: what the MMAs
    // take is then uniform over the warp.
    const uint32_t lead = elect_one() ? 1u : 0u;
    uint32_t it = 0, tc = 0;
    bool ok = true;
    for (int L = blockIdx.x; L < total && ok; L += gridDim.x, ++tc) {
      const Tile t = decode_tile<BM>(sched, args, L);
      const int n_kb = __shfl_sync(0xffffffffu, t.kb1 - t.kb0, 0);
      const uint32_t idesc = R::kSwap ? idesc_mx_e2m1_e4m3(128, BM)
                                      : idesc_mx_e4m3_e2m1(128, MODE == kGateUp ? 256 : bn, 0);
      if (R::kSwap) {
        // two accumulators apart from each other: this one's last tile has been read
        ok = __all_sync(0xffffffffu, mbar_wait(&tshared[tc & 1u], ((tc >> 1) & 1u) ^ 1u, abort_flag));
      } else if (tc > 0) {
        // the previous tile's epilogue has read the shared columns (and so has
        // finished the tile before, whose accumulator this one takes)
        ok = __all_sync(0xffffffffu, mbar_wait(&tshared[0], (tc - 1) & 1u, abort_flag));
      }
      if (!ok) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + ((tc & 1u) ? kAccSecond : 0);
      for (int i = 0; i < n_kb; ++i, ++it) {
        const uint32_t s = it % S, set = it % kScaleSets;
        ok = __all_sync(0xffffffffu, mbar_wait2(&full[s], (it / S) & 1u, &sfull[set], (it / kScaleSets) & 1u,
                                                abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = sw128_desc(smem_u32(sA + s * R::A_BYTES), 16, 1024);
        const uint64_t bd = sw128_desc(smem_u32(sB + s * B_BYTES), 16, 1024);
        const uint32_t sfa = tmem_base + kScaleCol + set * 12;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // 32 bytes of K further each: 2 in the descriptors' 16-byte units
          const uint32_t id = idesc | idesc_mx_scale_byte(kk), acc = (i > 0 || kk > 0) ? 1u : 0u;
          if (!R::kSwap) {
            umma_mxf8f6f4_if(lead, d_tmem, ad + 2 * kk, bd + 2 * kk, id, sfa, sfa + 4, acc);
          } else {
            umma_mxf8f6f4_if(lead, d_tmem, bd + 2 * kk, ad + 2 * kk, id, sfa + 4, sfa, acc);
            umma_mxf8f6f4_if(lead, d_tmem + BM, bd + 2 * kk + B_HALF / 16, ad + 2 * kk, id, sfa + 8, sfa, acc);
          }
        }
        umma_commit_if(lead, &empty[s]);
      }
      if (ok) umma_commit_if(lead, &tfull[tc & 1u]);
    }
    if (!ok) {
      if (lead) flag_error(args.err, MOE_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
    if (lead && it > 0) {
      // all MMAs must finish before TMEM and shared memory are released
      umma_commit(drain);
      mbar_wait(drain, 0, nullptr, 100000000ull);
    }
    __syncwarp();
  } else if (warp >= 6) {
    // ---------------------------------------------------------------- scales
    // On a path of their own beside the operands' ring: loads of kGroup K blocks
    // at a time (one lane of the first warp), and each block's 12 columns to its
    // TMEM set, all four lane quarters holding the same 32 lanes, one warp each.
    // (Moved by tcgen05.cp from the MMA warp, they stalled the MMAs.)  A set is
    // free when the MMAs four K blocks back are done.
    const int q = warp & 3;
    const bool loader = warp == 6 && lane == 0;
    uint32_t it = 0, grp = 0, issued = 0;
    bool ok = true;
    // tile and K block of the next group to load
    int lL = blockIdx.x, lkb = 0;
    Tile lt = {};
    if (lL < total) {
      lt = decode_tile<BM>(sched, args, lL);
      lkb = lt.kb0;
    }
    const uint64_t keep = policy_evict_last();
    auto load_groups = [&](uint32_t upto) {  // loader: groups below `upto`, their slots being free
      while (issued < upto && lL < total) {
        const uint32_t slot = issued % kGroupSlots;
        if (issued >= (uint32_t)kGroupSlots &&
            !mbar_wait(&gfree[slot], (issued / kGroupSlots - 1) & 1u, abort_flag))
          return false;
        const int n = min(kGroup, lt.kb1 - lkb);
        const uint32_t bytes = (uint32_t)n * 512;
        const int64_t eb = (int64_t)lt.e * args.nb_scales;
        const int64_t nb0 = eb + (MODE == kGateUp ? lt.nt : lt.nt * bn / 128);
        // a down tile of 128 columns has one block of scales, taken twice
        const int64_t second = MODE != kGateUp && bn > 128 ? (int64_t)args.num_kb * 512 : 0;
        const uint8_t* sa = args.a_scales + ((int64_t)lt.mtile * args.num_kb + lkb) * 512;
        const uint8_t* sb0 = args.b_scales0 + (nb0 * args.num_kb + lkb) * 512;
        const uint8_t* sb1 = MODE == kGateUp ? args.b_scales1 + (nb0 * args.num_kb + lkb) * 512
                                             : sb0 + second;
        uint8_t* g = sG + slot * GROUP_BYTES;
        mbar_arrive_expect_tx(&gfull[slot], 3 * bytes);
        bulk_load(g, sa, bytes, &gfull[slot], keep);
        bulk_load(g + kGroup * 512, sb0, bytes, &gfull[slot], keep);
        bulk_load(g + 2 * kGroup * 512, sb1, bytes, &gfull[slot], keep);
        ++issued;
        lkb += n;
        if (lkb >= lt.kb1) {
          lL += gridDim.x;
          if (lL < total) {
            lt = decode_tile<BM>(sched, args, lL);
            lkb = lt.kb0;
          }
        }
      }
      return true;
    };
    if (loader) ok = load_groups(kGroupSlots - 1);
    for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
      const Tile t = decode_tile<BM>(sched, args, L);
      for (int kb = t.kb0; kb < t.kb1 && ok; kb += kGroup, ++grp) {
        const uint32_t slot = grp % kGroupSlots;
        bool go = !loader || load_groups(grp + kGroupSlots);
        go = go && mbar_wait(&gfull[slot], (grp / kGroupSlots) & 1u, abort_flag);
        ok = __all_sync(0xffffffffu, go);
        if (!ok) break;
        const uint4* f = reinterpret_cast<const uint4*>(sG + slot * GROUP_BYTES) + lane;
        const int n = min(kGroup, t.kb1 - kb);
        for (int j = 0; j < n; ++j, ++it) {
          const uint32_t set = it % kScaleSets;
          uint4 va = f[j * 32], vb = f[kGroup * 32 + j * 32], vc = f[2 * kGroup * 32 + j * 32];
          // A tile that starts inside a 128-row block of scales (32 rows, or channels,
          // to a word): its first word goes to the first column, since the MMA takes
          // scales from columns at multiples of 4 (another column faulted).
          if (BM == 32) {
            const uint32_t rows32 = t.in_mtile / 32;
            va.x = rows32 == 0 ? va.x : (rows32 == 1 ? va.y : (rows32 == 2 ? va.z : va.w));
          } else if (BM == 64) {
            va.x = t.in_mtile == 0 ? va.x : va.z;
            va.y = t.in_mtile == 0 ? va.y : va.w;
          } else if (MODE == kDownSum && (t.nt * bn) % 128 != 0) {  // 192 columns from the middle of a block
            vb.x = vb.z;
            vb.y = vb.w;
            vb.z = vc.x;
            vb.w = vc.y;
            vc.x = vc.z;
            vc.y = vc.w;
          }
          if (it >= (uint32_t)kScaleSets) {
            const uint32_t done = it - kScaleSets;
            ok = __all_sync(0xffffffffu, mbar_wait(&empty[done % S], (done / S) & 1u, abort_flag));
            if (!ok) break;
          }
          tc_fence_after();
          const uint32_t dst = tmem_base + kScaleCol + set * 12 + ((uint32_t)(q * 32) << 16);
          tmem_st4(dst, va);
          tmem_st8(dst + 4, vb, vc);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull[set]);
        }
        if (ok && lane == 0) mbar_arrive(&gfree[slot]);
      }
    }
    if (!ok) {
      if (lane == 0) flag_error(args.err, MOE_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
    if (loader) {
      // drain, as the producer does
      const uint32_t first = issued > (uint32_t)kGroupSlots ? issued - kGroupSlots : 0u;
      for (uint32_t j = first; j < issued; ++j)
        mbar_wait(&gfull[j % kGroupSlots], (j / kGroupSlots) & 1u, nullptr, 100000000ull);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const int r = q * 32 + lane;
    uint32_t tc = 0;
    for (int L = blockIdx.x; L < total; L += gridDim.x, ++tc) {
      const Tile t = decode_tile<BM>(sched, args, L);
      const uint32_t buf = tc & 1u;
      if (!mbar_wait(&tfull[buf], (tc >> 1) & 1u, abort_flag)) {
        if (lane == 0) flag_error(args.err, MOE_DEVERR_TIMEOUT);
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      if (R::kSwap) {
        // lane = channel, column = row, 32 rows at a time
        const uint32_t tacc = tmem_base + (buf ? kAccSecond : 0) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
        for (int j0 = 0; j0 < BM; j0 += 32) {
          uint32_t v[2][32];
          tmem_ld32(tacc + j0, v[0]);
          tmem_ld32(tacc + BM + j0, v[1]);
          tmem_wait_ld();
          if (j0 + 32 >= BM) {
            tc_fence_before();
            mbar_arrive(&tshared[buf]);
          }
          const int n = t.rows - j0;  // rows of this batch, all above 31 alike
          if (n <= 0) continue;
          if (MODE == kGateUp) {
            uint8_t* dst = args.h + (int64_t)(t.m0 + j0) * args.ld + t.nt * 128 + r;
            uint8_t* sc = args.h_scales + ((int64_t)t.mtile * (args.ld / 128) + t.nt) * 512;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (j >= n) break;
              // the warp's 32 channels are the block
              const float h = silu_mul_fast(__uint_as_float(v[0][j]), __uint_as_float(v[1][j]));
              const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu);
              const int x = mx_exponent<8, kMxTopE4m3>(m);
              const bool bad = m >= 0x7f800000u;
              dst[j * args.ld] = bad ? 0x7f : (uint8_t)e4m3x2(h * mx_inverse(x), 0.f);
              if (lane == 0) sc[mx_scale_at(t.in_mtile + j0 + j, q)] = bad ? 255 : (uint8_t)(x + 127);
            }
          } else {
            const float mine = lane < n && args.row_scale ? __ldg(args.row_scale + t.m0 + j0 + lane) : 1.0f;
            float* dst = args.out + ((int64_t)t.split * args.rows_alloc + t.m0 + j0) * args.ld + t.nt * 256 + r;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (j >= n) break;
              const float s1 = __shfl_sync(0xffffffffu, mine, j);
              dst[j * args.ld] = s1 * __uint_as_float(v[0][j]);
              dst[j * args.ld + 128] = s1 * __uint_as_float(v[1][j]);
            }
          }
        }
        continue;
      }
      if (q * 32 >= t.rows) {  // a warp without rows reads nothing
        mbar_arrive(&tshared[0]);
        continue;
      }
      const bool valid = r < t.rows;
      const int row = t.m0 + r;
      const uint32_t tacc = tmem_base + (buf ? kAccSecond : 0) + ((uint32_t)(q * 32) << 16);
      // The shared columns first (the first accumulator's last 48, the second's
      // first 48: two chunks of 32), then the release: the next tile's MMAs wait
      // for nothing but these two loads.
      const int last = bn / 32 - 1;
      uint32_t early[2][32];
      const uint32_t tshare = MODE == kGateUp ? tacc + (buf ? 0 : 128) : tacc;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = buf ? i : last - i;
        tmem_ld32(tshare + c * 32, early[i]);
      }
      tmem_wait_ld();
      tmem_regs_ready(early[0]);
      tmem_regs_ready(early[1]);
      tc_fence_before();
      mbar_arrive(&tshared[0]);
      if (MODE == kGateUp) {
        uint32_t scales = 0;
        uint8_t* dst = args.h + (int64_t)row * args.ld + t.nt * 128;
        auto finish = [&](int c, const uint32_t (&g)[32], const uint32_t (&u)[32]) {
          float h[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) h[k] = silu_mul_fast(__uint_as_float(g[k]), __uint_as_float(u[k]));
          uint32_t codes[8];
          scales |= mx8_block(h, codes) << (8 * c);
          if (valid) {
            __stcs(reinterpret_cast<uint4*>(dst + c * 32), make_uint4(codes[0], codes[1], codes[2], codes[3]));
            __stcs(reinterpret_cast<uint4*>(dst + c * 32 + 16), make_uint4(codes[4], codes[5], codes[6], codes[7]));
          }
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = buf ? i : 3 - i;
          uint32_t other[32];  // gate beside the early up columns, or up beside the early gate columns
          tmem_ld32(tacc + (buf ? 128 : 0) + c * 32, other);
          tmem_wait_ld();
          if (buf)
            finish(c, early[i], other);
          else
            finish(c, other, early[i]);
        }
#pragma unroll 1
        for (int i = 2; i < 4; ++i) {
          const int c = buf ? i : 3 - i;
          uint32_t g[32], u[32];
          tmem_ld32(tacc + c * 32, g);
          tmem_ld32(tacc + 128 + c * 32, u);
          tmem_wait_ld();
          finish(c, g, u);
        }
        if (valid)
          *reinterpret_cast<uint32_t*>(args.h_scales + ((int64_t)t.mtile * (args.ld / 128) + t.nt) * 512 +
                                       mx_scale_at(t.in_mtile + r, 0)) = scales;
      } else {
        int64_t drow = (int64_t)t.split * args.rows_alloc + row;
        bool store = valid;
        if (MODE == kDownSum && valid) {
          const int tok = __ldg(args.perm + row);
          if (tok < 0 || (int64_t)tok >= args.n_tok) {
            flag_error(args.err, MOE_DEVERR_SLOT_INDEX);
            store = false;
          }
          drow = tok;
        }
        const float sc = (store && args.row_scale) ? __ldg(args.row_scale + row) : 1.0f;
        float* dst = args.out + (store ? drow : 0) * args.ld + t.nt * bn;
        // Sums: the 4-column pieces of eight rows change places among eight lanes
        // first, so that an instruction adds whole 128-byte lines of four rows and
        // not 16 bytes of 32 (T 4096, d 6144, f 8192: 349 against 381 us; whole
        // sectors in lane pairs 447, 64 bytes in fours 372).
        constexpr int kTurns = MODE == kDownSum ? 3 : 0, kRows = 1 << kTurns;
        float* dst_of[kRows];  // rows of this lane's group; NULL: not stored
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          dst_of[j] = reinterpret_cast<float*>(__shfl_sync(
              0xffffffffu, store ? reinterpret_cast<unsigned long long>(dst) : 0ull, (lane & ~(kRows - 1)) | j));
        auto finish = [&](int c, const uint32_t (&v)[32]) {
          float4 p[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            p[k] = make_float4(sc * __uint_as_float(v[4 * k]), sc * __uint_as_float(v[4 * k + 1]),
                               sc * __uint_as_float(v[4 * k + 2]), sc * __uint_as_float(v[4 * k + 3]));
          // piece k of lane l goes to piece (k, low bits of l) of lane (l, low bits of k)
#pragma unroll
          for (int s = 0; s < kTurns; ++s) {
            const bool odd = (lane >> s) & 1;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (k >> s & 1) continue;
              const int o = k | 1 << s;
              float4 x = odd ? p[k] : p[o];
              x.x = __shfl_xor_sync(0xffffffffu, x.x, 1 << s);
              x.y = __shfl_xor_sync(0xffffffffu, x.y, 1 << s);
              x.z = __shfl_xor_sync(0xffffffffu, x.z, 1 << s);
              x.w = __shfl_xor_sync(0xffffffffu, x.w, 1 << s);
              if (odd)
                p[k] = x;
              else
                p[o] = x;
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float* row_dst = dst_of[k & (kRows - 1)];
            if (!row_dst) continue;
            float4* d4 = reinterpret_cast<float4*>(row_dst + c * 32 + 4 * ((k & ~(kRows - 1)) | (lane & (kRows - 1))));
            if (MODE == kDownSum)
              atomicAdd(d4, p[k]);
            else
              *d4 = p[k];
          }
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) finish(buf ? i : last - i, early[i]);
#pragma unroll 1
        for (int i = 2; i <= last; ++i) {
          const int c = buf ? i : last - i;
          uint32_t v[32];
          tmem_ld32(tacc + c * 32, v);
          tmem_wait_ld();
          finish(c, v);
        }
      }
      tc_fence_before();
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// y[r, :] = sum over p of parts[p][r, :] in order, rows from offsets[0] to offsets[8].
__global__ void __launch_bounds__(256) mx4_sum_parts_kernel(const float4* __restrict__ parts, int n_parts,
                                                           const int32_t* __restrict__ offsets, int64_t max_rows,
                                                           int64_t row_vec, float4* __restrict__ y) {
  pdl_wait();
  const int64_t first = offsets[0];
  int64_t n = offsets[kE];
  if (first < 0 || n > max_rows) n = 0;
  for (int64_t i = first * row_vec + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n * row_vec;
       i += (int64_t)gridDim.x * blockDim.x) {
    float4 a = __ldg(parts + i);
    for (int p = 1; p < n_parts; ++p) {
      const float4 b = __ldg(parts + p * max_rows * row_vec + i);
      a.x += b.x;
      a.y += b.y;
      a.z += b.z;
      a.w += b.w;
    }
    y[i] = a;
  }
}

// out[t, :] = the token's kept slots' rows (slot 0 first), each the sum of its
// partials in order, rounded to bf16: moe_combine with weights_applied = 1, one
// float4 a thread, so that a few tokens fill the device (a block per token took
// 17 us for 32 tokens of 6144, the time of its chain of loads).
__global__ void __launch_bounds__(256) mx4_combine_kernel(const float4* __restrict__ parts, int n_parts, int64_t stride,
                                                         const int32_t* __restrict__ slot_of, int64_t n,
                                                         int64_t row_vec, int64_t max_slot, uint2* __restrict__ out,
                                                         int* err) {
  pdl_wait();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int64_t t = i / row_vec, v = i - t * row_vec;
  const int2 sl = __ldg(reinterpret_cast<const int2*>(slot_of) + t);
  const int s[2] = {sl.x, sl.y};
  float4 r[2][kMaxDownSplits];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const bool on = s[j] >= 0 && s[j] < max_slot;
    if (s[j] >= max_slot || s[j] < -1) flag_error(err, MOE_DEVERR_SLOT_INDEX);
#pragma unroll
    for (int p = 0; p < kMaxDownSplits; ++p)
      r[j][p] = on && p < n_parts ? __ldg(parts + p * stride + s[j] * row_vec + v) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float4 y = r[j][0];
#pragma unroll
    for (int p = 1; p < kMaxDownSplits; ++p) {
      y.x += r[j][p].x;
      y.y += r[j][p].y;
      y.z += r[j][p].z;
      y.w += r[j][p].w;
    }
    a.x += y.x;
    a.y += y.y;
    a.z += y.z;
    a.w += y.w;
  }
  out[i] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
}

template <int MODE, int BM>
cudaError_t launch_mx_tiles(const CUtensorMap& a, const CUtensorMap& a32, const CUtensorMap& b0, const CUtensorMap& b1,
                            const MxArgs& args, cudaStream_t s, const Ctx& ctx) {
  auto kern = mx4_gemm_kernel<MODE, BM>;
  constexpr int smem = Ring<BM>::SMEM_BYTES;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(ctx.num_sms), dim3(kThreads), smem, s, no_extra_attr(), a, a32, b0, b1, args);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Row tiles that hold an expert's rows at once: 32 where it gets up to 24 on the
// average, 64 up to 48, else 128.  Gate/up, d 6144, f 32768: T 96 263 us with
// tiles of 32 against 323 with 128; T 128 337 with 32 (a second tile reads the
// weights again), 282 with 64, 328 with 128; T 192 415, 293, 331.
template <int MODE>
cudaError_t launch_mx(const CUtensorMap& a, const CUtensorMap& a32, const CUtensorMap& b0, const CUtensorMap& b1,
                      const MxArgs& args, cudaStream_t s, const Ctx& ctx) {
  if constexpr (MODE != kDownSum) {
    if (args.rows_alloc <= 24 * kE) return launch_mx_tiles<MODE, 32>(a, a32, b0, b1, args, s, ctx);
    if (args.rows_alloc <= 48 * kE) return launch_mx_tiles<MODE, 64>(a, a32, b0, b1, args, s, ctx);
  }
  return launch_mx_tiles<MODE, 128>(a, a32, b0, b1, args, s, ctx);
}

// [rows, K] e4m3 codes, box of 128 columns x box_rows rows.
bool map_rows8(CUtensorMap* m, const void* base, int64_t rows, int64_t K, uint32_t box_rows) {
  const uint64_t dims[2] = {(uint64_t)K, (uint64_t)rows};
  const uint64_t str[1] = {(uint64_t)K};
  const uint32_t box[2] = {BK, box_rows};
  return encode_tmap_dtype(m, base, 2, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_UINT8);
}

// [E, N, K / 2] packed e2m1 codes, box of 128 codes x `channels`, spread to 16 bytes per 16 codes.
bool map_codes4(CUtensorMap* m, const void* base, int E, int64_t N, int64_t K, uint32_t channels) {
  const uint64_t dims[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)E};
  const uint64_t str[2] = {(uint64_t)K / 2, (uint64_t)N * K / 2};
  const uint32_t box[3] = {BK, channels, 1};
  return encode_tmap_dtype(m, base, 3, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B);
}

MxArgs base_args(const moe_config_t& c, const int32_t* offsets, const Ctx& ctx) {
  MxArgs a = {};
  a.offsets = offsets;
  a.rows_alloc = slot_rows(c);
  a.splits = 1;
  a.n_tok = c.T;
  a.err = ctx.err;
  return a;
}

}  // namespace

int64_t mx_row_tiles(const moe_config_t& c) { return slot_rows(c) / 128 + c.E; }

// K splits of the down pass where at most 64 rows an expert are expected (the
// weight-streaming sizes): the smallest count that leaves the last wave of tiles
// at least 97% full, assuming min(8, rows) experts in use; else the fullest.
int mx4_down_splits(const moe_config_t& c, int num_sms) {
  const int64_t rows = slot_rows(c);
  if (rows > 64 * (int64_t)c.E) return 1;
  const int64_t base = (rows < c.E ? rows : c.E) * (c.d / 256), kb = c.f / BK;
  int best = 1;
  double best_eff = 0.0;
  for (int sp = 1; sp <= kMaxDownSplits && sp <= kb; ++sp) {
    const int64_t tiles = base * sp, waves = (tiles + num_sms - 1) / num_sms;
    const double eff = (double)tiles / (double)(waves * num_sms);
    if (eff > best_eff + 1e-9) {
      best_eff = eff;
      best = sp;
    }
    if (eff >= 0.97) break;
  }
  return best;
}

cudaError_t launch_mx4_gate_up(const moe_config_t& c, const uint8_t* x8, const uint8_t* x_scales,
                               const int32_t* offsets, const Mx4Weights& gate, const Mx4Weights& up, uint8_t* h8,
                               uint8_t* h_scales, cudaStream_t s, const Ctx& ctx) {
  const int64_t rows = slot_rows(c);
  if (rows == 0) return cudaSuccess;
  CUtensorMap ta, ta32, tg, tu;
  if (!map_rows8(&ta, x8, rows, c.d, 128) || !map_rows8(&ta32, x8, rows, c.d, 32) ||
      !map_codes4(&tg, gate.codes, c.E, c.f, c.d, 128) || !map_codes4(&tu, up.codes, c.E, c.f, c.d, 128))
    return cudaErrorInvalidValue;
  MxArgs a = base_args(c, offsets, ctx);
  a.n_tiles = (int)(c.f / 128);
  a.bn = 128;
  a.num_kb = (int)(c.d / BK);
  a.a_scales = x_scales;
  a.b_scales0 = gate.scales;
  a.b_scales1 = up.scales;
  a.nb_scales = (int)(c.f / 128);
  a.h = h8;
  a.h_scales = h_scales;
  a.ld = c.f;
  return launch_mx<kGateUp>(ta, ta32, tg, tu, a, s, ctx);
}

cudaError_t launch_mx4_down(const moe_config_t& c, const uint8_t* h8, const uint8_t* h_scales, const int32_t* offsets,
                            const Mx4Weights& down, const float* row_scale, const int32_t* perm, float* out, int splits,
                            cudaStream_t s, const Ctx& ctx) {
  const int64_t rows = slot_rows(c);
  if (rows == 0) return cudaSuccess;
  CUtensorMap ta, ta32, td;
  MxArgs a = base_args(c, offsets, ctx);
  a.bn = perm ? tile_columns(c, c.d, {256, 192, 128}, ctx.num_sms) : 256;
  if (!map_rows8(&ta, h8, rows, c.f, 128) || !map_rows8(&ta32, h8, rows, c.f, 32) ||
      !map_codes4(&td, down.codes, c.E, c.d, c.f, a.bn % 128 == 0 ? 128 : 64))
    return cudaErrorInvalidValue;
  a.n_tiles = (int)(c.d / a.bn);
  a.num_kb = (int)(c.f / BK);
  a.splits = splits;
  a.a_scales = h_scales;
  a.b_scales0 = down.scales;
  a.nb_scales = (int)(c.d / 128);
  a.out = out;
  a.ld = c.d;
  a.row_scale = row_scale;
  a.perm = perm;
  if (perm) return launch_mx<kDownSum>(ta, ta32, td, td, a, s, ctx);
  return launch_mx<kDownParts>(ta, ta32, td, td, a, s, ctx);
}

cudaError_t launch_mx4_sum_parts(const moe_config_t& c, const float* parts, int n_parts, const int32_t* offsets,
                                 float* y, cudaStream_t s, const Ctx& ctx) {
  const int64_t rows = slot_rows(c);
  if (rows == 0) return cudaSuccess;
  const cudaError_t e = launch_pdl(mx4_sum_parts_kernel, dim3(ctx.num_sms * 4), dim3(256), 0, s, no_extra_attr(),
                                   reinterpret_cast<const float4*>(parts), n_parts, offsets, rows, c.d / 4,
                                   reinterpret_cast<float4*>(y));
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_mx4_combine(const moe_config_t& c, const float* parts, int n_parts, const int32_t* slot_of, void* out,
                               cudaStream_t s, const Ctx& ctx) {
  const int64_t n = c.T * c.d / 4;
  if (n == 0) return cudaSuccess;
  const cudaError_t e = launch_pdl(mx4_combine_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                                   no_extra_attr(), reinterpret_cast<const float4*>(parts), n_parts,
                                   slot_rows(c) * c.d / 4, slot_of, n, c.d / 4, slot_rows(c),
                                   static_cast<uint2*>(out), ctx.err);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
