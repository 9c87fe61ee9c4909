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
#include "stream4.hpp"

namespace nvfp4 {

namespace {

constexpr int kI4Waves = 4;
#ifndef I4_NT1
#define I4_NT1 4
#define I4_SC1 1
#endif
// 16-row weight tiles per wavefront, and 128-k chunks per step of its pipeline
constexpr int i4_tiles(int mt) { return mt == 1 ? I4_NT1 : 2; }
constexpr int i4_super(int mt) { return mt == 1 ? I4_SC1 : 1; }
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
// of 128, or one group per row).  A wavefront owns NT tiles of 16 weight rows; `splitk` of
// the workgroup's four share them, taking every splitk-th run of SC chunks, and
// their partial sums are added in wavefront order.
template <int MT, int NG, bool ZP>
__global__ __launch_bounds__(64 * kI4Waves) void int4_gemm_kernel(Int4Args a) {
  constexpr int NT = i4_tiles(MT), SC = i4_super(MT);
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
    u32x4 x[4][MT];
  };
  auto load = [&](int c, Chunk& ch) {
    const int k0 = kI4Chunk * c;
    const int j = NG == 1 ? k0 / a.group : NG * c;      // first group of the chunk
    const bool whole = k0 + kI4Chunk <= K;              // uniform over the wavefront
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        ch.x[s][i] = xin[i] && k0 + 32 * s < K ? *reinterpret_cast<const u32x4*>(xrow[i] + k0 + 32 * s)
                                               : u32x4{0u, 0u, 0u, 0u};
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

  auto compute = [&](Chunk& ch) {
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
        xa[i] = reorder_x(ch.x[s][i]);
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
      if (SC * sp + q < nchunks) compute(ch[q]);
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

// ---------------------------------------------------------------------------
// Up to 16 activation rows (stream4.hpp's scheme).  Wavefront w of a workgroup
// keeps the x fragments of its NC chunks of 256 k, and the workgroup streams the
// 16-row tiles that it owns past them.  The workgroup's threads fetch a tile's
// scales (and zero points) together, whole rows of them, D + 1 tiles ahead into
// registers, and leave them in LDS one tile ahead as float32 words whose four
// low bits, zero in any bf16 or f16 value, hold the zero point.  The
// wavefronts' sums of a tile meet in LDS (two buffers, one barrier a tile).  K
// beyond W NC chunks is taken in phases over the same tiles, whose sums wait in
// LDS meanwhile.
// ---------------------------------------------------------------------------
template <int NC, int NG, bool ZP, int D>
__global__ __launch_bounds__(NC == 1 ? 1024 : 768) void int4_stream_kernel(Int4Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds8[];
  constexpr int SI = (NC * NG + 1) / 2;                 // scales per thread and tile
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int W = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int K = a.K, N = a.N;
  const int64_t pitch = K >> 1;
  const int nchunks = (K + kSt4Chunk - 1) / kSt4Chunk;
  const int tiles = (N + 15) >> 4;
  const int t0 = (int)((int64_t)tiles * blockIdx.x / gridDim.x), t1 = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  const int phases = (nchunks + W * NC - 1) / (W * NC);
  uint8_t* const ring = lds8 + wave * (D * NC * kSt4Bytes);
  float* const red = reinterpret_cast<float*>(lds8 + W * (D * NC * kSt4Bytes));   // [2][W][256]
  uint32_t* const scl = reinterpret_cast<uint32_t*>(red + 2 * W * 256);           // [2][16][a.scale_pitch]
  float* const held = reinterpret_cast<float*>(scl + 2 * 16 * a.scale_pitch);     // [t1 - t0][256], several phases
  const int spitch = a.scale_pitch;

  for (int ph = 0; ph < phases; ++ph) {
    const int c0 = (ph * W + wave) * NC;                // this wavefront's first chunk
    // the phase's groups: [j0, j0 + gn) of each row
    const int j0 = ph * W * NC * kSt4Chunk / a.group;
    const int gn = min(a.groups, ((ph + 1) * W * NC * kSt4Chunk + a.group - 1) / a.group) - j0;
    int srow[SI], scol[SI];
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      const int it = tid + i * blockDim.x;
      srow[i] = it / gn;
      scol[i] = it - srow[i] * gn;
    }
    // loads are unconditional (clamped): a branch would make the compiler wait
    uint32_t sv[D][SI], zv[D][SI];
    auto load_scales = [&](int t, int slot) {
      const int last = min(15, N - 1 - 16 * t);
#pragma unroll
      for (int i = 0; i < SI; ++i) {
        const int row = 16 * t + min(srow[i], last);
        sv[slot][i] = a.scales[(int64_t)row * a.groups + j0 + scol[i]];
        if (ZP) zv[slot][i] = (uint32_t)a.zeros[(int64_t)(row >> 3) * a.groups + j0 + scol[i]];
      }
    };
    auto store_scales = [&](int t, int slot) {
#pragma unroll
      for (int i = 0; i < SI; ++i) {
        if (srow[i] < 16) {
          uint32_t w = __float_as_uint(scale_value(sv[slot][i], a.scale_f16));
          if (ZP) w |= (zv[slot][i] >> (4 * (srow[i] & 7))) & 15u;
          scl[((t & 1) * 16 + srow[i]) * spitch + scol[i]] = w;
        }
      }
    };
    auto copy_tile = [&](int t, int slot) {
      const int tc = min(t, t1 - 1);                    // past the last: a repeat, never read
#pragma unroll
      for (int q = 0; q < NC; ++q)
        st4_copy(a.packed + (int64_t)16 * tc * pitch, pitch, N - 1 - 16 * tc, c0 + q,
                 ring + (slot * NC + q) * kSt4Bytes, lane);
    };

    // the scales travel one tile ahead of the copies, so that the wait for a
    // tile's copies covers the next tile's scales
    if (t0 < t1) {
      load_scales(t0, 0);
      store_scales(t0, 0);
#pragma unroll
      for (int d = 0; d < D; ++d) {
        load_scales(min(t0 + d + 1, t1 - 1), d);
        copy_tile(t0 + d, d);
      }
    }
    // x fragments, in the order of the codes: MFMA step s of sub-chunk h (128 k)
    // is k = 32 s + 8 g + [0, 8), or k = 32 g + 8 s + [0, 8) where the whole
    // sub-chunk lies in one group and the words stay where they are
    bf16x8 xa[NC][2][4];
    f32x4 base[NC][2];
    const u32x4 one_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    const bf16x8 one = __builtin_bit_cast(bf16x8, one_bits);
    {
      const uint16_t* const xrow = a.x + (int64_t)min(r, a.M - 1) * K;
#pragma unroll
      for (int q = 0; q < NC; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const int k = kSt4Chunk * (c0 + q) + 128 * h + (NG == 1 ? 32 * g + 8 * s : 32 * s + 8 * g);
            xa[q][h][s] = reorder_x(k < K ? *reinterpret_cast<const u32x4*>(xrow + k) : u32x4{0u, 0u, 0u, 0u});
          }
          if (NG == 1) {                                // sum x over the sub-chunk, once
            base[q][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 4; ++s) base[q][h] = mfma_i4(xa[q][h][s], one, base[q][h]);
#pragma unroll
            for (int v = 0; v < 4; ++v) base[q][h][v] *= ZP ? -1.0f : -136.0f;
          }
        }
    }
    st4_barrier();

    auto step = [&](int t, int slot) {
      // the copies of tile t are older than those of the D - 1 tiles after it
      __builtin_amdgcn_s_waitcnt(st4_vm((D - 1) * (2 * NC + SI * (ZP ? 2 : 1))));
      __asm__ volatile("" ::: "memory");
      u32x4 w[NC][2];
      uint32_t sw[NC][2][NG];
#pragma unroll
      for (int q = 0; q < NC; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[q][h] = st4_read(ring + (slot * NC + q) * kSt4Bytes, r, 4 * h + g);
          const int k = kSt4Chunk * (c0 + q) + 128 * h;
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const int j = NG == 1 ? k / a.group : NG * (k / 128) + i;
            // beyond the row's groups the activations are zero
            sw[q][h][i] = scl[((t & 1) * 16 + r) * spitch + min(j - j0, gn - 1)];
          }
        }
      __builtin_amdgcn_s_waitcnt(kSt4Lgkm0);            // the region may now be refilled
      __asm__ volatile("" ::: "memory");
      if (t + 1 < t1) store_scales(t + 1, slot);
      load_scales(min(t + D + 1, t1 - 1), slot);
      copy_tile(t + D, slot);

      f32x4 total = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < NC; ++q) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (NG == 1) {
            const uint32_t sb = sw[q][h][0];
            f32x4 acc = base[q][h];
            if (ZP) {
              const float off = 128.0f + (float)(sb & 15u);
#pragma unroll
              for (int v = 0; v < 4; ++v) acc[v] *= off;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) acc = mfma_i4(xa[q][h][s], codes_bf16(w[q][h][s]), acc);
            const float sc = __uint_as_float(ZP ? sb & ~15u : sb);
#pragma unroll
            for (int v = 0; v < 4; ++v) total[v] = __builtin_fmaf(sc, acc[v], total[v]);
          } else {
            transpose4(w[q][h]);
            f32x4 acc, ones;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              constexpr int kSteps = 4 / NG;
              const bool fresh = s % kSteps == 0;
              const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
              ones = mfma_i4(xa[q][h][s], one, fresh ? zero : ones);
              acc = mfma_i4(xa[q][h][s], codes_bf16(w[q][h][s]), fresh ? zero : acc);
              if (s % kSteps == kSteps - 1) {
                const uint32_t sb = sw[q][h][s / kSteps];
                const float sc = __uint_as_float(ZP ? sb & ~15u : sb);
                const float off = 128.0f + (ZP ? (float)(sb & 15u) : 8.0f);
#pragma unroll
                for (int v = 0; v < 4; ++v) total[v] = __builtin_fmaf(sc, __builtin_fmaf(-off, ones[v], acc[v]), total[v]);
              }
            }
          }
        }
      }
      *reinterpret_cast<f32x4*>(red + ((t & 1) * W + wave) * 256 + 4 * lane) = total;
      st4_barrier();
      // element 4 l + v is lane l's v: row 4 (l / 16) + v of x, weight row l % 16
      for (int i = tid; i < 256; i += blockDim.x) {
        const int m = 4 * (i >> 6) + (i & 3), n = 16 * t + ((i >> 2) & 15);
        if (m >= a.M || n >= N) continue;
        const float* const part = red + (t & 1) * W * 256 + i;
        float sum = 0.0f;
        for (int v = 0; v < W; v += 4) {                // four reads at a time, added in order
          float q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = part[min(v + e, W - 1) * 256];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += v + e < W ? q[e] : 0.0f;
        }
        if (phases > 1) {
          float* const h = held + (t - t0) * 256 + i;
          if (ph > 0) sum += *h;
          if (ph + 1 < phases) {
            *h = sum;
            continue;
          }
        }
        if (a.bias) sum += __uint_as_float((uint32_t)a.bias[n] << 16);
        a.y[(int64_t)m * N + n] = __builtin_bit_cast(uint16_t, (__bf16)sum);
      }
    };
    for (int t = t0; t < t1; t += D) {
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (t + d < t1) step(t + d, d);
    }
    __builtin_amdgcn_s_waitcnt(st4_vm(0));              // trailing copies land before the regions are used again
    __syncthreads();
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

namespace {

constexpr int kI4Depth = 3;                  // tiles in flight per wavefront

template <int NC>
const void* int4_stream(int ng, bool zp) {
  constexpr int D = kI4Depth;
  if (zp)
    return ng == 4   ? (const void*)int4_stream_kernel<NC, 4, true, D>
           : ng == 2 ? (const void*)int4_stream_kernel<NC, 2, true, D>
                     : (const void*)int4_stream_kernel<NC, 1, true, D>;
  return ng == 4   ? (const void*)int4_stream_kernel<NC, 4, false, D>
         : ng == 2 ? (const void*)int4_stream_kernel<NC, 2, false, D>
                   : (const void*)int4_stream_kernel<NC, 1, false, D>;
}

// M <= 16: the wavefronts (at most 16) and their chunks (1 or 2) that take K in the
// fewest phases, then with the fewest idle chunk slots.
hipError_t launch_int4_stream(Int4Args a, int ng, hipStream_t stream) {
  const int64_t nchunks = (a.K + kSt4Chunk - 1) / kSt4Chunk;
  int nc = 1, waves = 1;
  int64_t best = INT64_MAX;
  for (int c = 1; c <= 2; ++c) {
    const int64_t most = c == 1 ? 16 : 11;              // LDS: D c 2 KB a wavefront beside the sums
    const int64_t phases = (nchunks + most * c - 1) / (most * c);
    const int64_t w = (nchunks + phases * c - 1) / (phases * c);
    const int64_t cost = phases * 1000000 + (w * c * phases - nchunks) * 1000 + c;
    if (cost < best) {
      best = cost;
      nc = c;
      waves = (int)w;
    }
  }
  const int64_t phases = (nchunks + waves * nc - 1) / (waves * nc);
  const int dev = current_device();
  const int64_t tiles = ((int64_t)a.N + 15) / 16;
  // groups of a phase: at most its k / group, one more where they straddle
  a.scale_pitch = (int)(std::min<int64_t>(a.groups, (int64_t)waves * nc * kSt4Chunk / a.group + 2) | 1);
  int64_t lds = (int64_t)waves * (kI4Depth * nc * kSt4Bytes + 2048) + 128 * a.scale_pitch;
  const int per_cu = (int)std::max<int64_t>(1, std::min<int64_t>(16 / waves, 160 * 1024 / (lds + 1024)));
  int64_t grid = std::min<int64_t>(tiles, (int64_t)device_cus(dev) * per_cu);
  if (phases > 1) {                                     // the held sums of a workgroup's tiles fit beside
    const int64_t room = (158 * 1024 - lds) / 1024;
    grid = std::max<int64_t>(grid, (tiles + room - 1) / room);
    lds += (tiles + grid - 1) / grid * 1024;
  }
  const void* fn = nc == 1 ? int4_stream<1>(ng, a.zeros != nullptr) : int4_stream<2>(ng, a.zeros != nullptr);
  if (lds > 65536) {
    const hipError_t e = ensure_dynamic_lds(fn, dev, (int)lds);
    if (e != hipSuccess) return e;
  }
  return launch_kernel_lds(fn, dim3((unsigned)grid), dim3(64 * waves), (size_t)lds, stream, a);
}

}  // namespace

hipError_t launch_int4_gemm(Int4Args a, hipStream_t stream) {
  const int ng = a.group == 32 && a.K > 32 ? 4 : a.group == 64 && a.K > 64 ? 2 : 1;
  if (a.M <= 16 && a.K <= (1 << 27)) return launch_int4_stream(a, ng, stream);
  const int mt = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
  // K split over 1, 2 or 4 wavefronts, so that the wavefronts fill the GPU
  // (eight for each of 256 compute units)
  const int64_t row_groups = ((int64_t)a.N + 16 * i4_tiles(mt) - 1) / (16 * i4_tiles(mt));
  const int64_t nsuper = (a.K + i4_super(mt) * kI4Chunk - 1) / (i4_super(mt) * kI4Chunk);
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
