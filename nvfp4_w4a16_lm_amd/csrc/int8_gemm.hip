// 8-bit integer weights and activations (gfx950): one scale for each token and
// each channel.
//
//   quantizer   s = max(max_k |a| / 127, 1e-12),  q = round(127 a / max_k |a|), nearest even;
//               with a NaN or an infinity in the row s = NaN and q = 0, so that all its products are NaN
//   product     y[m, n] = bf16( sx[m] sw[n] sum_k xq[m, k] wq[n, k] + bias[n] )
//
// The sums are exact in 32 bits: |q| <= 128 and K < 2^17.  Measured, quantizer and product: 1 x
// 128256 x 4096 93 us (5.7 TB/s, HBM), 16 x 151936 x 5120 143 us (5.5 TB/s), 33 x 32003 x 2080 20 us (17 the product:
// a start and seventeen steps), 4096 x 28672 x 4096 440 us (2.2 POPS, power).  K is not split: few columns leave compute
// units idle (1 x 4096 x 14336, 32 workgroups of 112 steps: 46 us, floor 11.5; 128 x 4096 x 4096 27 us, floor 3.7).
#include "dense_tile.hpp"

namespace nvfp4 {

// ---------------------------------------------------------------------------
// int8_quant_rows_kernel: a workgroup per row, the row's first 8192 elements
// kept in registers between the maximum and the rounding.
//
// The codes are those of the exact ratio 127 a / amax: 127 a is exact in float32 (a has 8 bits), the
// division rounds once, a ratio on a border k + 1/2 is itself a float32 and so comes out exactly, and any
// other is at least 2^-17 of itself away from a border (|127 a / b - (2 k + 1) / 2| is a nonzero
// multiple of 1 / (2 b) up to powers of two, b < 256).  a / s instead would miss borders: half the
// maximum is on one in every row.
// ---------------------------------------------------------------------------
constexpr int kQ8Threads = 256, kQ8Keep = 4;

__global__ __launch_bounds__(kQ8Threads) void int8_quant_rows_kernel(const uint16_t* __restrict__ a, int K,
                                                                     uint8_t* __restrict__ q,
                                                                     float* __restrict__ scales) {
  __shared__ uint32_t part[kQ8Threads / 64];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const u32x4* const src = reinterpret_cast<const u32x4*>(a + row * K);
  const int pieces = K / 8;
  u32x4 keep[kQ8Keep];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < kQ8Keep; ++i) {
    const int p = tid + i * kQ8Threads;
    keep[i] = p < pieces ? src[p] : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = pk_max_u16(mx, keep[i][e] & 0x7FFF7FFFu);
  }
  for (int p = tid + kQ8Keep * kQ8Threads; p < pieces; p += kQ8Threads) {
    const u32x4 v = src[p];
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = pk_max_u16(mx, v[e] & 0x7FFF7FFFu);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mx = pk_max_u16(mx, (uint32_t)__shfl_xor((int)mx, d, 64));
  if ((tid & 63) == 0) part[tid >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQ8Threads / 64; ++w) mx = pk_max_u16(mx, part[w]);
  // the bits of magnitudes order as the magnitudes, infinity and then the NaN above all: such a row shows in amax
  const float amax = __uint_as_float(max(mx & 0xFFFFu, mx >> 16) << 16);
  const bool finite = amax < INFINITY;
  const float s = finite ? fmaxf(__fdiv_rn(amax, 127.0f), 1e-12f) : NAN;
  if (tid == 0) scales[row] = s;
  // where the scale is the smallest one, a / s; where 127 a could overflow, everything 2^-8 as large
  const bool least = s == 1e-12f, large = amax > 0x1p100f;
  const float factor = least ? 1.0f : large ? 127.0f * 0x1p-8f : 127.0f;
  const float over = least ? s : large ? amax * 0x1p-8f : amax;
  auto code = [&](float v) __attribute__((always_inline)) {
    return (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(v * factor, over)), -127.0f), 127.0f) & 0xFFu;
  };
  auto codes = [&](u32x4 v) __attribute__((always_inline)) {
    if (!finite) return make_uint2(0, 0);
    uint2 o;
    o.x = code(bf16_lo(v[0])) | code(bf16_hi(v[0])) << 8 | code(bf16_lo(v[1])) << 16 | code(bf16_hi(v[1])) << 24;
    o.y = code(bf16_lo(v[2])) | code(bf16_hi(v[2])) << 8 | code(bf16_lo(v[3])) << 16 | code(bf16_hi(v[3])) << 24;
    return o;
  };
  uint2* const dst = reinterpret_cast<uint2*>(q + row * K);
#pragma unroll
  for (int i = 0; i < kQ8Keep; ++i) {
    const int p = tid + i * kQ8Threads;
    if (p < pieces) dst[p] = codes(keep[i]);
  }
  for (int p = tid + kQ8Keep * kQ8Threads; p < pieces; p += kQ8Threads) dst[p] = codes(src[p]);
}

hipError_t launch_int8_quant_rows(const void* a, int64_t R, int64_t K, int8_t* q, float* scales, hipStream_t stream) {
  return launch_kernel((const void*)int8_quant_rows_kernel, dim3((unsigned)R), dim3(kQ8Threads), stream,
                       (const uint16_t*)a, (int)K, (uint8_t*)q, scales);
}

hipError_t launch_int8_gemm(const int8_t* xq, const float* sx, int64_t M, int64_t K, const int8_t* wq,
                            const float* sw, int64_t N, const void* bias, void* y, hipStream_t stream) {
  TileArgs a = {};
  a.p = (const uint8_t*)wq;
  a.q = (const uint8_t*)xq;
  a.p_pitch = a.q_pitch = K;
  a.p_rows = N;
  a.q_rows = M;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.splits = 1;
  a.k_split = 1 << 20;
  a.out = y;
  a.out_pitch = N;
  a.sx = sx;
  a.sw = sw;
  a.bias = (const uint16_t*)bias;
  return launch_tile<kTileInt8, false, false>(a, tile_size(M, N, (K + 127) / 128, 1), stream);
}

}  // namespace nvfp4
