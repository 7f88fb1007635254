// Microscaled 4-bit weights and 8-bit activation rows.
//
// quantize: w [E, K, N] bf16 (N contiguous) -> codes [E, N, K / 2] (K
// contiguous: the 4-bit operand of the block-scaled MMA has to be K-major) and
// scales in blocks of 128 channels x 128 K.  Bound by memory (2 + 0.53 bytes a
// weight): 6.3 TB/s for [8, 32768, 6144] (640 to 646 us), and 5.8 to 6.0 TB/s back
// (684 to 700 us; blocks that run along K instead of N took 749 us); on a box with
// slower DRAM the two take 1373 us together.  A block of 256 threads
// takes 128 K x 128 channels: a thread reads one 32-block of two channels (rows
// of 256 bytes across the block), so the largest magnitude needs no exchange,
// and the codes turn through shared memory into 64-byte runs.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace moe {
namespace {

constexpr int kRow = 80;  // bytes of a channel's 64 code bytes in shared memory (16-byte pieces, banks shifted)

__global__ void __launch_bounds__(256) quantize_mx4_kernel(const __nv_bfloat16* __restrict__ w, int64_t K, int64_t N,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint8_t s_codes[128 * kRow];
  __shared__ __align__(16) uint8_t s_scale[512];
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int64_t nb = blockIdx.x, kb = blockIdx.y, e = blockIdx.z;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(w + (e * K + kb * 128 + ty * 32) * N + nb * 128) + tx;
  uint32_t v[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = __ldcs(src + k * (N / 2));
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) m = max(m, (j == 0 ? v[k] << 16 : v[k] & 0xffff0000u) & 0x7fffffffu);
    const int x = mx_exponent<2, kMxTopE2m1>(m);
    const bool bad = m >= 0x7f800000u;
    const float inv = mx_inverse(x);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        f[k] = __uint_as_float(j == 0 ? v[8 * i + k] << 16 : v[8 * i + k] & 0xffff0000u) * inv;
      c[i] = bad ? 0u : e2m1x8(f);
    }
    const int n = 2 * tx + j;
    *reinterpret_cast<uint4*>(s_codes + n * kRow + ty * 16) = make_uint4(c[0], c[1], c[2], c[3]);
    s_scale[mx_scale_at(n, ty)] = bad ? 255 : (uint8_t)(x + 127);
  }
  __syncthreads();
  uint8_t* dst = codes + ((e * N + nb * 128) * K + kb * 128) / 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = threadIdx.x + 256 * i, n = p >> 2, q = p & 3;
    *reinterpret_cast<uint4*>(dst + n * (K / 2) + q * 16) = *reinterpret_cast<const uint4*>(s_codes + n * kRow + q * 16);
  }
  if (threadIdx.x < 32)
    reinterpret_cast<uint4*>(scales + ((e * (N / 128) + nb) * (K / 128) + kb) * 512)[threadIdx.x] =
        reinterpret_cast<const uint4*>(s_scale)[threadIdx.x];
}

// The same tiles back.  A thread decodes 8 K of 8 neighbouring channels and
// writes 16 bytes of each of the 8 rows of K, a row of the tile being 256 bytes
// of 16 threads (4-byte stores, two channels a thread, ran at 0.83 of the copy
// rate).  17 words a channel in shared memory: its reads meet four to a bank.
__global__ void __launch_bounds__(256) dequantize_mx4_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t K, int64_t N,
                                                            __nv_bfloat16* __restrict__ w) {
  __shared__ uint32_t s_codes[128 * 17];
  __shared__ __align__(16) uint8_t s_scale[512];
  const int64_t nb = blockIdx.x, kb = blockIdx.y, e = blockIdx.z;
  const uint8_t* src = codes + ((e * N + nb * 128) * K + kb * 128) / 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = threadIdx.x + 256 * i, n = p >> 2, q = p & 3;
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src + n * (K / 2) + q * 16));
    uint32_t* to = s_codes + n * 17 + q * 4;
    to[0] = v.x;
    to[1] = v.y;
    to[2] = v.z;
    to[3] = v.w;
  }
  if (threadIdx.x < 32)
    reinterpret_cast<uint4*>(s_scale)[threadIdx.x] =
        __ldcs(reinterpret_cast<const uint4*>(scales + ((e * (N / 128) + nb) * (K / 128) + kb) * 512) + threadIdx.x);
  __syncthreads();
  const int ng = threadIdx.x & 15, ks = threadIdx.x >> 4;  // channels 8 ng .. + 7, K 8 ks .. + 7
  uint32_t c[8];
  float sc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = 8 * ng + j;
    c[j] = s_codes[n * 17 + ks];
    const int b = s_scale[mx_scale_at(n, ks >> 2)];
    // 2^(b - 127), 2^-127 (b = 0) as the subnormal it is, 255 as NaN
    sc[j] = b == 255 ? __uint_as_float(0x7fc00000u) : (b == 0 ? 0x1p-127f : __uint_as_float((uint32_t)b << 23));
  }
  uint4* dst = reinterpret_cast<uint4*>(w + (e * K + kb * 128 + ks * 8) * N + nb * 128) + ng;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = pack_bf16x2(e2m1_value(c[2 * i] >> (4 * k)) * sc[2 * i], e2m1_value(c[2 * i + 1] >> (4 * k)) * sc[2 * i + 1]);
    __stcs(dst + k * (N / 8), make_uint4(o[0], o[1], o[2], o[3]));
  }
}

// Grouped rows to e4m3: row r of the codes, from offsets[0] to offsets[8], is src
// row r, or src[perm[r]] when perm is given.  A thread takes 8 values (16 bytes), four
// neighbours one 32-block, a warp 256 columns of a row at a time with four such
// pieces in flight; blockIdx.y shares the columns out, so that a few rows still
// spread over the SMs.  The scale of row r goes to the 512-byte block of its
// tile (row tiles of 128 start anew at each expert).
__global__ void __launch_bounds__(256) quantize_rows_mx8_kernel(const __nv_bfloat16* __restrict__ src,
                                                               const int32_t* __restrict__ perm, int64_t n_src,
                                                               const int32_t* __restrict__ offsets, int64_t max_rows,
                                                               int64_t K, uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales, int* err) {
  __shared__ int s_off[9], s_tile[9];
  pdl_wait();
  if (threadIdx.x == 0) {
    bool ok = true;
    int tile = 0, prev = 0, v[9];
#pragma unroll
    for (int k = 0; k <= 8; ++k) v[k] = offsets[k];
#pragma unroll
    for (int k = 0; k <= 8; ++k) {
      if (v[k] < prev || (int64_t)v[k] > max_rows) ok = false;
      if (k && ok) tile += (v[k] - prev + 127) / 128;
      s_off[k] = v[k];
      s_tile[k] = tile;
      prev = v[k];
    }
    if (!ok) {
      s_off[0] = s_off[8] = 0;
      flag_error(err, MOE_DEVERR_OFFSETS);
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int pieces = (int)(K / 256);
  const int per = (pieces + (int)gridDim.y - 1) / (int)gridDim.y;
  const int c_begin = (int)blockIdx.y * per, c_end = min(c_begin + per, pieces);
  const int rows = s_off[8], warps = (int)gridDim.x * 8;
  for (int r = s_off[0] + (int)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += warps) {
    int64_t sr = r;
    if (perm) {
      sr = __ldg(perm + r);
      if (sr < 0 || sr >= n_src) {
        if (lane == 0) flag_error(err, MOE_DEVERR_SLOT_INDEX);
        continue;
      }
    }
    int e = 0;
#pragma unroll
    for (int k = 1; k < 8; ++k)
      if (r >= s_off[k]) e = k;
    const int in_expert = r - s_off[e];
    const uint4* from = reinterpret_cast<const uint4*>(src + sr * K) + lane;
    uint2* to = reinterpret_cast<uint2*>(codes + (int64_t)r * K) + lane;
    uint8_t* sc = scales + (int64_t)(s_tile[e] + in_expert / 128) * (K / 128) * 512;
    for (int c0 = c_begin; c0 < c_end; c0 += 4) {
      uint4 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + i < c_end) q[i] = __ldg(from + (c0 + i) * 32);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + i;
        if (c >= c_end) break;
        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
        float v[8];
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[2 * k] = __uint_as_float(w[k] << 16);
          v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
          m = max(m, max(w[k] << 16 & 0x7fffffffu, w[k] & 0x7fff0000u));
        }
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int x = mx_exponent<8, kMxTopE4m3>(m);
        const float inv = mx_inverse(x);
        uint2 o = make_uint2(e4m3x2(v[0] * inv, v[1] * inv) | e4m3x2(v[2] * inv, v[3] * inv) << 16,
                             e4m3x2(v[4] * inv, v[5] * inv) | e4m3x2(v[6] * inv, v[7] * inv) << 16);
        const bool bad = m >= 0x7f800000u;
        if (bad) o = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        to[c * 32] = o;
        // the warp's 8 blocks are two words of four scales: lanes 0 and 16 write one each
        uint32_t byte = bad ? 255u : (uint32_t)(x + 127);
        byte |= __shfl_down_sync(0xffffffffu, byte, 4) << 8;
        byte |= __shfl_down_sync(0xffffffffu, byte, 8) << 16;
        if ((lane & 15) == 0)
          *reinterpret_cast<uint32_t*>(sc + (c * 2 + lane / 16) * 512 + mx_scale_at(in_expert, 0)) = byte;
      }
    }
  }
}

}  // namespace

cudaError_t launch_quantize_mx4(int E, const void* w, int64_t K, int64_t N, uint8_t* codes, uint8_t* scales,
                                cudaStream_t s) {
  dim3 grid((unsigned)(N / 128), (unsigned)(K / 128), (unsigned)E);  // neighbours on the same rows of w
  quantize_mx4_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(w), K, N, codes, scales);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_mx4(int E, const uint8_t* codes, const uint8_t* scales, int64_t K, int64_t N, void* w,
                                  cudaStream_t s) {
  dim3 grid((unsigned)(N / 128), (unsigned)(K / 128), (unsigned)E);  // neighbours on the same rows of w
  dequantize_mx4_kernel<<<grid, 256, 0, s>>>(codes, scales, K, N, static_cast<__nv_bfloat16*>(w));
  return cudaGetLastError();
}

cudaError_t launch_quantize_rows_mx8(const void* src, const int32_t* perm, int64_t n_src, const int32_t* offsets,
                                     int64_t max_rows, int64_t K, uint8_t* codes, uint8_t* scales, cudaStream_t s,
                                     const Ctx& ctx) {
  if (max_rows == 0) return cudaSuccess;
  const int64_t want = (max_rows + 7) / 8, cap = (int64_t)ctx.num_sms * 8;
  const unsigned gx = (unsigned)(want < cap ? want : cap);
  // columns in pieces of 256, shared out until there are two blocks an SM
  int64_t gy = 1;
  while (gy * 2 <= K / 256 && gx * gy < 2 * ctx.num_sms) gy *= 2;
  const cudaError_t e =
      launch_pdl(quantize_rows_mx8_kernel, dim3(gx, (unsigned)gy), dim3(256), 0, s, no_extra_attr(),
                 static_cast<const __nv_bfloat16*>(src), perm, n_src, offsets, max_rows, K, codes, scales, ctx.err);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
