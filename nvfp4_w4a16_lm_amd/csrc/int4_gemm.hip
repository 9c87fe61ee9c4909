// W4A16 product with int4 weights and group scales (gfx950), for few
// activation rows: y[m, n] = sum_j s[n, j] sum_{k in group j} x[m, k] (q[n, k] - z[n, j]) (+ bias).
//
// Layout (vLLM API docs, compressed_tensors.schemes, CompressedTensorsWNA16):
// eight codes per 32-bit word along K, low nibble first; scales [N, K / group]
// in bf16 or f16; zero points eight rows per word along N, or none (z = 8).
//
// A code q becomes the bf16 value 128 + q by one and-or (0x4300 | q: at
// exponent 2^7 the last mantissa bit is worth 1), two codes at a time: (w >> 4 i) & 0x000F000F
// holds codes i and i + 4, so the activations are taken in the same order
// (0, 4, 1, 5, ...).  The MFMA's A operand is x (16 rows), B is 16 weight rows, so
// a lane's accumulators all belong to its own weight row (lane % 16) and the
// row's scale is one value of that lane.  A product of x with a tile of ones
// gives sum x over the same k in the same places, and per group
//   total += s (acc - (128 + z) ones)
// in float32: every product is exact, the only roundings are float32 sums and
// that step.
//
// A lane (r, g) = (lane % 16, lane / 16) loads row r's codes of k = 128 c + 32 g + [0, 32)
// as 16 bytes.  Two permlane32 and two permlane16 swaps transpose the 4 x 4
// words among the four g, after which word s of lane (r, g) holds
// k = 128 c + 32 s + 8 g + [0, 8): an MFMA step covers 32 consecutive k and so lies in
// one group for every group size from 32.
#include <algorithm>

#include "nvfp4_device.hpp"
#include "nvfp4_launch.hpp"

namespace nvfp4 {

namespace {

constexpr int kI4Waves = 4;
constexpr int kI4NT = 2;                     // 16-row weight tiles per wavefront
// 128-k chunks per step of the pipeline: as many as the registers allow
constexpr int i4_super(int mt, int ng) { return mt == 1 && ng < 4 ? 4 : mt <= 2 ? 2 : 1; }
constexpr int kI4Chunk = 128;

struct __attribute__((packed, aligned(2))) Scale4A2 { uint2 v; };
struct __attribute__((packed, aligned(2))) Scale2A2 { uint32_t v; };
struct __attribute__((packed, aligned(4))) Zero4A4 { u32x4 v; };
struct __attribute__((packed, aligned(4))) Zero2A4 { uint2 v; };

__device__ __forceinline__ f32x4 mfma_i4(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 4 x 4 transpose of words among the lanes r, r + 16, r + 32, r + 48.
__device__ __forceinline__ void transpose4(u32x4& w) {
  uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
  auto p = __builtin_amdgcn_permlane32_swap(a, c, false, false);
  a = p[0];
  c = p[1];
  p = __builtin_amdgcn_permlane32_swap(b, d, false, false);
  b = p[0];
  d = p[1];
  p = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = p[0];
  b = p[1];
  p = __builtin_amdgcn_permlane16_swap(c, d, false, false);
  w = u32x4{a, b, p[0], p[1]};
}

// Eight codes -> 128 + code in bf16, codes (0, 4, 1, 5, 2, 6, 3, 7).
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8, o);
}

// Eight activations in that order.
__device__ __forceinline__ bf16x8 reorder_x(u32x4 d) {
  u32x4 o;
  o[0] = __builtin_amdgcn_perm(d[2], d[0], 0x05040100u);
  o[1] = __builtin_amdgcn_perm(d[2], d[0], 0x07060302u);
  o[2] = __builtin_amdgcn_perm(d[3], d[1], 0x05040100u);
  o[3] = __builtin_amdgcn_perm(d[3], d[1], 0x07060302u);
  return __builtin_bit_cast(bf16x8, o);
}

__device__ __forceinline__ float scale_value(uint32_t bits16, bool f16) {
  const uint16_t h = (uint16_t)bits16;
  return f16 ? (float)__builtin_bit_cast(_Float16, h) : __uint_as_float((uint32_t)h << 16);
}

}  // namespace

// NG: scales per 128-k chunk (4, 2: groups of 32, 64; 1: groups of a multiple
// of 128, or one group per row).  A wavefront owns 32 weight rows; `splitk` of
// the workgroup's four share them, taking every splitk-th run of SC chunks, and
// their partial sums are added in wavefront order.
template <int MT, int NG, bool ZP>
__global__ __launch_bounds__(64 * kI4Waves) void int4_gemm_kernel(Int4Args a) {
  constexpr int NT = kI4NT, SC = i4_super(MT, NG);
  __shared__ float red[kI4Waves][NT * MT * 4][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int mb = blockIdx.y * 16 * MT;
  const int splitk = a.splitk, rg = wave / splitk, ph = wave - rg * splitk;
  const int nb = (blockIdx.x * (kI4Waves / splitk) + rg) * 16 * NT;     // this wavefront's first row
  const int K = a.K, N = a.N;
  const int nchunks = (K + kI4Chunk - 1) / kI4Chunk;
  const int nsuper = (nchunks + SC - 1) / SC;

  const uint8_t* wrow[NT];
  const uint16_t* srow[NT];
  const uint32_t* zrow[NT];
  int zshift[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = min(nb + 16 * t + r, N - 1);
    wrow[t] = a.packed + (int64_t)n * (K >> 1) + 16 * g;
    srow[t] = a.scales + (int64_t)n * a.groups;
    zrow[t] = ZP ? a.zeros + (int64_t)(n >> 3) * a.groups : nullptr;
    zshift[t] = 4 * (n & 7);
  }
  const uint16_t* xrow[MT];
  bool xin[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = mb + 16 * i + r;
    xin[i] = m < a.M;
    xrow[i] = a.x + (int64_t)min(m, a.M - 1) * K + 8 * g;
  }

  struct Chunk {
    u32x4 w[NT];
    uint32_t s[NT][(NG + 1) / 2];            // scales, two to a word
    uint32_t z[NT][NG];
  };
  auto load = [&](int c, Chunk& ch) {
    const int k0 = kI4Chunk * c;
    const int j = NG == 1 ? k0 / a.group : NG * c;      // first group of the chunk
    const bool whole = k0 + kI4Chunk <= K;              // uniform over the wavefront
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (whole) {
        ch.w[t] = load_stream16(wrow[t] + (k0 >> 1));
        if (NG == 4) {
          const uint2 v = reinterpret_cast<const Scale4A2*>(srow[t] + j)->v;
          ch.s[t][0] = v.x;
          ch.s[t][(NG + 1) / 2 - 1] = v.y;
        } else if (NG == 2) {
          ch.s[t][0] = reinterpret_cast<const Scale2A2*>(srow[t] + j)->v;
        } else {
          ch.s[t][0] = srow[t][j];
        }
        if (ZP) {
          if (NG == 4) {
            const u32x4 v = reinterpret_cast<const Zero4A4*>(zrow[t] + j)->v;
#pragma unroll
            for (int i = 0; i < NG; ++i) ch.z[t][i] = v[i];
          } else if (NG == 2) {
            const uint2 v = reinterpret_cast<const Zero2A4*>(zrow[t] + j)->v;
            ch.z[t][0] = v.x;
            ch.z[t][NG - 1] = v.y;
          } else {
            ch.z[t][0] = zrow[t][j];
          }
        }
      } else {
        ch.w[t] = k0 + 32 * g < K ? load_stream16(wrow[t] + (k0 >> 1)) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < (NG + 1) / 2; ++i) ch.s[t][i] = 0;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const bool in = j + i < a.groups && k0 < K;
          ch.s[t][i / 2] |= in ? (uint32_t)srow[t][j + i] << (16 * (i & 1)) : 0u;
          if (ZP) ch.z[t][i] = in ? zrow[t][j + i] : 0u;
        }
      }
    }
  };

  f32x4 total[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < MT; ++i) total[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 one_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const bf16x8 one = __builtin_bit_cast(bf16x8, one_bits);

  auto compute = [&](int c, Chunk& ch) {
    const int k0 = kI4Chunk * c;
    u32x4 xv[4][MT];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        xv[s][i] = xin[i] && k0 + 32 * s < K ? *reinterpret_cast<const u32x4*>(xrow[i] + k0 + 32 * s)
                                             : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int t = 0; t < NT; ++t) transpose4(ch.w[t]);
    f32x4 acc[NT][MT], ones[MT];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      constexpr int kSteps = 4 / NG;                    // steps per group
      const bool fresh = s % kSteps == 0;
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      bf16x8 xa[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        xa[i] = reorder_x(xv[s][i]);
        ones[i] = mfma_i4(xa[i], one, fresh ? zero : ones[i]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bf16x8 wb = codes_bf16(ch.w[t][s]);
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[t][i] = mfma_i4(xa[i], wb, fresh ? zero : acc[t][i]);
      }
      if (s % kSteps == kSteps - 1) {
        const int q = s / kSteps;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float sc = scale_value(ch.s[t][q / 2] >> (16 * (q & 1)), a.scale_f16);
          const float off = 128.0f + (ZP ? (float)((ch.z[t][q] >> zshift[t]) & 15u) : 8.0f);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              total[t][i][v] = __builtin_fmaf(sc, __builtin_fmaf(-off, ones[i][v], acc[t][i][v]), total[t][i][v]);
        }
      }
    }
  };

  Chunk cur[SC], next[SC];
  auto load_super = [&](int sp, Chunk* ch) {
#pragma unroll
    for (int q = 0; q < SC; ++q)
      if (SC * sp + q < nchunks) load(SC * sp + q, ch[q]);
  };
  auto compute_super = [&](int sp, Chunk* ch) {
#pragma unroll
    for (int q = 0; q < SC; ++q)
      if (SC * sp + q < nchunks) compute(SC * sp + q, ch[q]);
  };
  if (ph < nsuper) load_super(ph, cur);
  for (int sp = ph; sp < nsuper; sp += 2 * splitk) {
    if (sp + splitk < nsuper) load_super(sp + splitk, next);
    compute_super(sp, cur);
    if (sp + splitk >= nsuper) break;
    if (sp + 2 * splitk < nsuper) load_super(sp + 2 * splitk, cur);
    compute_super(sp + splitk, next);
  }

  if (splitk > 1) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[wave][(t * MT + i) * 4 + v][lane] = total[t][i][v];
    __syncthreads();
    if (ph != 0) return;
    for (int q = 1; q < splitk; ++q)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) total[t][i][v] += red[wave + q][(t * MT + i) * 4 + v][lane];
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = nb + 16 * t + r;
    if (n >= N) continue;
    const float b = a.bias ? __uint_as_float((uint32_t)a.bias[n] << 16) : 0.0f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int m = mb + 16 * i + 4 * g + v;
        if (m < a.M) a.y[(int64_t)m * N + n] = __builtin_bit_cast(uint16_t, (__bf16)(total[t][i][v] + b));
      }
  }
}

namespace {

template <int MT, int NG>
const void* int4_kernel(bool zp) {
  return zp ? (const void*)int4_gemm_kernel<MT, NG, true> : (const void*)int4_gemm_kernel<MT, NG, false>;
}

template <int MT>
const void* int4_kernel(int ng, bool zp) {
  return ng == 4 ? int4_kernel<MT, 4>(zp) : ng == 2 ? int4_kernel<MT, 2>(zp) : int4_kernel<MT, 1>(zp);
}

}  // namespace

hipError_t launch_int4_gemm(Int4Args a, hipStream_t stream) {
  const int ng = a.group == 32 && a.K > 32 ? 4 : a.group == 64 && a.K > 64 ? 2 : 1;
  const int mt = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
  // K split over 1, 2 or 4 wavefronts, so that the wavefronts fill the GPU
  // (eight for each of 256 compute units)
  const int64_t row_groups = ((int64_t)a.N + 16 * kI4NT - 1) / (16 * kI4NT);
  const int64_t nsuper = (a.K + i4_super(mt, ng) * kI4Chunk - 1) / (i4_super(mt, ng) * kI4Chunk);
  int splitk = 1;
  while (splitk < kI4Waves && row_groups * splitk < 4096 && 2 * splitk <= nsuper) splitk *= 2;
  a.splitk = splitk;
  const int64_t per = kI4Waves / splitk;
  const dim3 grid((unsigned)((row_groups + per - 1) / per), (unsigned)((a.M + 16 * mt - 1) / (16 * mt)));
  const void* fn = mt == 1   ? int4_kernel<1>(ng, a.zeros != nullptr)
                   : mt == 2 ? int4_kernel<2>(ng, a.zeros != nullptr)
                             : int4_kernel<4>(ng, a.zeros != nullptr);
  return launch_kernel(fn, grid, dim3(64 * kI4Waves), stream, a);
}

}  // namespace nvfp4
