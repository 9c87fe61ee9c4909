// W4A16 product with int4 weights and group scales (gfx950), for few
// activation rows: y[m, n] = sum_j s[n, j] sum_{k in group j} x[m, k] (q[n, k] - z[n, j]) (+ bias).
//
// Layout (vLLM API docs, compressed_tensors.schemes, CompressedTensorsWNA16):
// eight codes per 32-bit word along K, low nibble first; scales [N, K / group]
// in bf16 or f16; zero points eight rows per word along N, or none (z = 8).
//
// A code q becomes the bf16 value 16 + q by one and-or (0x4180 | q << 3: at
// exponent 2^4 the fourth mantissa bit from below is worth 1), two codes at a time: (w >> (4 i - 3)) &
// 0x00780078 holds codes i and i + 4, so the activations are taken in the same order
// (0, 4, 1, 5, ...).  The offset goes out of the sums again, at the price of the bits
// that a sum of 31 |x| needs beyond one of 8 or 15 |x|, one or two; 128 + q, which
// saves the first pair's shift (1 to 3 % of the time), loses four or five, and overflows
// from |x| = 2^121 on.  The MFMA's A operand is x (16 rows), B is 16 weight rows, so
// a lane's accumulators all belong to its own weight row (lane % 16) and the
// row's scale is one value of that lane.  The offset 16 + z goes through the
// MFMA as well: where a group has 128 k or more, x times a tile of ones, once,
// gives sum x in the accumulator's places, and -(16 + z) sum x starts each group's
// sum; with smaller groups a tile of the constant -(16 + z) (exact in bf16) is
// multiplied along.  Per group then total += s acc in float32: every product is
// exact, the only roundings are float32 sums and that step.
//
// A lane (r, g) = (lane % 16, lane / 16) reads row r's codes of k = 128 c + 32 g + [0, 32)
// as 16 bytes; its word s and those of the other three g make an MFMA step of
// 32 k out of the 128.  Where a group is smaller than 128, two permlane32 and
// two permlane16 swaps first transpose the 4 x 4 words among the four g, so that
// step s covers the consecutive k = 128 c + 32 s + [0, 32) and lies in one group.
#include <algorithm>

#include "int4_groups.hpp"
#include "nvfp4_device.hpp"
#include "nvfp4_launch.hpp"
#include "stream4.hpp"

namespace nvfp4 {

namespace {

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

// Codes i and i + 4 of a word shifted down by 4 i - 3.  The constants are hidden from the
// compiler in a scalar and a vector register, or it spends two instructions
// (v_and_or_b32 takes one scalar operand and no literal).
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t mask = 0x00780078u, one = 0x41804180u;
  __asm__("" : "+s"(mask));
  __asm__("" : "+v"(one));
  return (w & mask) | one;
}

__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {
  return code_pair(i == 0 ? w << 3 : w >> (4 * i - 3));
}

// Eight codes -> 16 + code in bf16, codes (0, 4, 1, 5, 2, 6, 3, 7).
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = code_pair(w, i);
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

// ---------------------------------------------------------------------------
// One or two activation rows: whole rows of the weight past the wavefront, 64
// consecutive 16-byte segments (32 k each) a load, each lane always the same
// segments, so that its x stays in registers: no LDS, no barrier.  A code's
// bf16 16 + q goes into v_dot2_f32_bf16 (float32 sum of exact products) with its
// neighbour four codes on; a segment lies in one group.  Four rows a batch, the
// next batch on its way meanwhile.  VALU and HBM about balance.  128256 x 4096,
// M = 1, groups of 128: 46 us (5.9 TB/s).  Against the streamed form below, random
// codes: 128256 x 4096 55 and 67 us; 8192 x 2048 4.7 and 8.4; 128256 x 8192 110 and 125.
// ---------------------------------------------------------------------------
template <int MR, int SEG, bool ZP>
__global__ __launch_bounds__(256) void int4_dot_kernel(Int4Args a) {
  const int lane = threadIdx.x & 63, wave = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = gridDim.x * 4, N = a.N, K = a.K;
  const int nseg = K >> 5;
  u32x4 xr[MR][SEG][4];
  float sumx[MR][SEG];
  int seg[SEG], grp[SEG];
#pragma unroll
  for (int j = 0; j < SEG; ++j) {
    seg[j] = min(lane + 64 * j, nseg - 1);               // beyond the row: a repeat, against x = 0
    grp[j] = seg[j] * 32 / a.group;
  }
  struct Batch {
    u32x4 w[4][SEG];
    uint32_t s[4][SEG], z[4][SEG];
  };
  auto load = [&](int r0, Batch& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = min(r0 + i, N - 1);             // repeats are computed, not stored
      const uint8_t* const wp = a.packed + row * (K >> 1);
      const uint16_t* const sp = a.scales + row * a.groups;
      const uint32_t* const zp = ZP ? a.zeros + (row >> 3) * a.groups : nullptr;
#pragma unroll
      for (int j = 0; j < SEG; ++j) {
        b.w[i][j] = load_stream16(wp + (uint32_t)(16 * seg[j]));
        b.s[i][j] = sp[(uint32_t)grp[j]];
        if (ZP) b.z[i][j] = zp[(uint32_t)grp[j]];
      }
    }
  };
  auto compute = [&](int r0, const Batch& b) {
    float p[MR][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int m = 0; m < MR; ++m) p[m][i] = 0.0f;
#pragma unroll
      for (int j = 0; j < SEG; ++j) {
        float sc = scale_value(b.s[i][j], a.scale_f16);
        if (j == SEG - 1 && lane + 64 * j >= nseg) sc = 0.0f;   // lest an infinite scale meet x = 0
        const float off = ZP ? 16.0f + (float)((b.z[i][j] >> (4 * (min(r0 + i, N - 1) & 7))) & 15u) : 24.0f;
        float blk[MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) blk[m] = -off * sumx[m][j];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t word = b.w[i][j][q];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t c = code_pair(word, e);
#pragma unroll
            for (int m = 0; m < MR; ++m) {
              const uint32_t xe = xr[m][j][q][e];
              blk[m] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, c), __builtin_bit_cast(bf16x2, xe),
                                                       blk[m], false);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < MR; ++m) p[m][i] = __builtin_fmaf(sc, blk[m], p[m][i]);
      }
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      const float tot = wave_sum4(p[m], lane);
      const int row = r0 + ((lane >> 5) & 1) * 2 + ((lane >> 4) & 1);
      if ((lane & 15) == 0 && row < N && m < a.M) {
        const float bias = a.bias ? __uint_as_float((uint32_t)a.bias[row] << 16) : 0.0f;
        a.y[(int64_t)m * N + row] = __builtin_bit_cast(uint16_t, (__bf16)(tot + bias));
      }
    }
  };
  Batch b0, b1;
  const int first = 4 * wave, step = 4 * waves;
  if (first < N) load(first, b0);
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int j = 0; j < SEG; ++j) {
      const bool in = lane + 64 * j < nseg;
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(a.x + (int64_t)min(m, a.M - 1) * K + 32 * seg[j] + 8 * q);
        const u32x4 o = __builtin_bit_cast(u32x4, reorder_x(v));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = in ? o[e] : 0u;
          xr[m][j][q][e] = w;
          s += bf16_lo(w) + bf16_hi(w);
        }
      }
      sumx[m][j] = s;
    }
  for (int r0 = first; r0 < N; r0 += 2 * step) {
    const bool more = r0 + step < N;
    if (more) load(r0 + step, b1);
    compute(r0, b0);
    if (!more) break;
    if (r0 + 2 * step < N) load(r0 + 2 * step, b0);
    compute(r0 + step, b1);
  }
}

// ---------------------------------------------------------------------------
// stream4.hpp's scheme for 16 MT activation rows.  Wavefront w of a workgroup
// keeps the x fragments of its NC chunks of 256 k, and the workgroup streams the
// 16-row tiles that it owns past them.  The workgroup's threads fetch a tile's
// scales (and zero points) together, whole rows of them, D + 1 tiles ahead into
// registers, and leave them in LDS one tile ahead as float32 words whose four
// low bits, zero in any bf16 or f16 value, hold the zero point.  The
// wavefronts' sums of a tile meet in LDS (two buffers and one barrier a tile up
// to 16 rows; one buffer and two barriers beyond, where LDS is short).  K
// beyond W NC chunks is taken in phases over the same tiles, whose sums wait in
// LDS meanwhile.  NG: scales per 128 k (4, 2: groups of 32, 64; 1: groups of a
// multiple of 128, or one group per row).  Up to 16 rows HBM bounds it (16 x 151936 x
// 5120, zero points: 86 us, 4.8 TB/s; weights loaded to registers in the MFMA's layout,
// four lanes a row: 216), beyond that, where few weight rows leave this form the
// only one that fills the card, the unpacking and the sums through LDS (64 x 8000 x
// 8192: 52 us).
// ---------------------------------------------------------------------------
// Wavefronts per workgroup: the x fragments take 32 MT NC registers of each lane.
// Sum buffers, and tiles in flight per wavefront: beyond 16 rows the LDS that the
// sums held from phase to phase need is worth more (M = 64, 128256 x 4096, before
// the tile kernel took that size: 210 us with two buffers and three tiles, 155 so).
constexpr int i4_buffers(int mt) { return mt == 1 ? 2 : 1; }
constexpr int i4_depth(int mt) { return mt == 1 ? 3 : 2; }
constexpr int i4_max_waves(int mt, int nc) { return mt * nc == 1 ? 16 : mt * nc == 2 ? 11 : 8; }

template <int MT, int NC, int NG, bool ZP, int D>
__global__ __launch_bounds__(MT * NC == 1 ? 1024 : MT * NC == 2 ? 768 : 512) void int4_stream_kernel(Int4Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds8[];
  constexpr int SI = (NC * NG + 1) / 2;                 // scales per thread and tile
  constexpr int RB = i4_buffers(MT);
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
  float* const red = reinterpret_cast<float*>(lds8 + W * (D * NC * kSt4Bytes));   // [RB][W][MT][256]
  uint32_t* const scl = reinterpret_cast<uint32_t*>(red + RB * W * MT * 256);      // [2][16][a.scale_pitch]
  float* const bias = reinterpret_cast<float*>(scl + 2 * 16 * a.scale_pitch);     // [t1 - t0][16]
  float* const held = bias + 16 * a.tiles_per_block;                              // [t1 - t0][MT][256], several phases
  const int spitch = a.scale_pitch;
  // every bias of the workgroup's rows, now: a load in the loop would wait for the copies
  for (int i = tid; i < 16 * (t1 - t0); i += blockDim.x)
    bias[i] = a.bias && 16 * t0 + i < N ? __uint_as_float((uint32_t)a.bias[16 * t0 + i] << 16) : 0.0f;
  const int mb = 16 * MT * blockIdx.y;

  for (int ph = 0; ph < phases; ++ph) {
    const int c0 = (ph * W + wave) * NC;                // this wavefront's first chunk
    // the phase's groups: [j0, j0 + gn) of each row
    const I4Groups of = i4_groups(ph * W * NC * kSt4Chunk, W * NC * kSt4Chunk, K, a.group);
    const int j0 = of.first, gn = of.count;
    int srow[SI], scol[SI];
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      const int it = tid + i * blockDim.x;
      srow[i] = it / gn;
      scol[i] = it - srow[i] * gn;
    }
    // loads are unconditional (clamped): a branch would make the compiler wait
    uint32_t sv[D + 1][SI], zv[D + 1][SI];              // the last entry: the first tile's
    auto load_scales = [&](int t, int slot) {
      const int last = min(15, N - 1 - 16 * t);
      const uint16_t* const sb = a.scales + (int64_t)16 * t * a.groups + j0;
      const uint32_t* const zb = ZP ? a.zeros + (int64_t)2 * t * a.groups + j0 : nullptr;
#pragma unroll
      for (int i = 0; i < SI; ++i) {
        const int row = min(srow[i], last);
        sv[slot][i] = sb[(uint32_t)(row * a.groups + scol[i])];
        if (ZP) zv[slot][i] = zb[(uint32_t)((row >> 3) * a.groups + scol[i])];
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
      load_scales(t0, D);
#pragma unroll
      for (int d = 0; d < D; ++d) {
        load_scales(min(t0 + d + 1, t1 - 1), d);
        copy_tile(t0 + d, d);
      }
      store_scales(t0, D);
    }
    // x fragments, in the order of the codes: MFMA step s of sub-chunk h (128 k)
    // is k = 32 s + 8 g + [0, 8), or k = 32 g + 8 s + [0, 8) where the whole
    // sub-chunk lies in one group and the words stay where they are
    bf16x8 xa[NC][2][4][MT];
    f32x4 base[NC][2][MT];
    const u32x4 one_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    const bf16x8 one = __builtin_bit_cast(bf16x8, one_bits);
    {
#pragma unroll
      for (int q = 0; q < NC; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const uint16_t* const xrow = a.x + (int64_t)min(mb + 16 * i + r, a.M - 1) * K;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const int k = kSt4Chunk * (c0 + q) + 128 * h + (NG == 1 ? 32 * g + 8 * s : 32 * s + 8 * g);
              xa[q][h][s][i] = reorder_x(k < K ? *reinterpret_cast<const u32x4*>(xrow + k) : u32x4{0u, 0u, 0u, 0u});
            }
            if (NG == 1) {                              // sum x over the sub-chunk, once
              f32x4 b = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int s = 0; s < 4; ++s) b = mfma_i4(xa[q][h][s][i], one, b);
#pragma unroll
              for (int v = 0; v < 4; ++v) base[q][h][i][v] = b[v] * (ZP ? -1.0f : -24.0f);
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
            // beyond the row's groups the activations are zero; 0, lest an infinite scale meet them
            const uint32_t word = scl[((t & 1) * 16 + r) * spitch + min(j - j0, gn - 1)];
            sw[q][h][i] = j - j0 < gn ? word : 0u;
          }
        }
      __builtin_amdgcn_s_waitcnt(kSt4Lgkm0);            // the region may now be refilled
      __asm__ volatile("" ::: "memory");
      if (t + 1 < t1) store_scales(t + 1, slot);
      load_scales(min(t + D + 1, t1 - 1), slot);
      copy_tile(t + D, slot);

      f32x4 total[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) total[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < NC; ++q) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (NG > 1) transpose4(w[q][h]);
          f32x4 acc[MT];
          const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
          if (NG == 1) {
            const float off = 16.0f + (float)(sw[q][h][0] & 15u);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int v = 0; v < 4; ++v) acc[i][v] = ZP ? off * base[q][h][i][v] : base[q][h][i][v];
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            constexpr int kSteps = 4 / NG;              // MFMA steps per group
            const bool fresh = NG > 1 && s % kSteps == 0;
            const bf16x8 wb = codes_bf16(w[q][h][s]);
            // small groups: -(16 + z) of the lane's row as a tile of its own, exact in bf16
            const uint32_t ob = ZP ? (0xC180u | (sw[q][h][s / kSteps] & 15u) << 3) * 0x10001u : 0xC1C0C1C0u;
            const u32x4 obits = {ob, ob, ob, ob};
            const bf16x8 off = __builtin_bit_cast(bf16x8, obits);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              acc[i] = mfma_i4(xa[q][h][s][i], wb, fresh ? zero : acc[i]);
              if (NG > 1) acc[i] = mfma_i4(xa[q][h][s][i], off, acc[i]);
            }
            if (s % kSteps == kSteps - 1) {
              const uint32_t sb = sw[q][h][s / kSteps];
              const float sc = __uint_as_float(ZP ? sb & ~15u : sb);
#pragma unroll
              for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) total[i][v] = __builtin_fmaf(sc, acc[i][v], total[i][v]);
            }
          }
        }
      }
      const int buf = RB == 2 ? t & 1 : 0;
      if (RB == 1) st4_barrier();                       // the tile before has been summed
#pragma unroll
      for (int i = 0; i < MT; ++i)
        *reinterpret_cast<f32x4*>(red + ((buf * W + wave) * MT + i) * 256 + 4 * lane) = total[i];
      st4_barrier();
      // element 4 l + v is lane l's v: row 4 (l / 16) + v of x, weight row l % 16
      for (int i = tid; i < 256 * MT; i += blockDim.x) {
        const int m = mb + 16 * (i >> 8) + 4 * ((i >> 6) & 3) + (i & 3), n = 16 * t + ((i >> 2) & 15);
        if (m >= a.M || n >= N) continue;
        const float* const part = red + buf * W * MT * 256 + i;
        float sum = 0.0f;
        for (int v = 0; v < W; v += 4) {                // four reads at a time, added in order
          float q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = part[min(v + e, W - 1) * MT * 256];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += v + e < W ? q[e] : 0.0f;
        }
        if (phases > 1) {
          float* const h = held + (t - t0) * MT * 256 + i;
          if (ph > 0) sum += *h;
          if (ph + 1 < phases) {
            *h = sum;
            continue;
          }
        }
        if (a.bias) sum += bias[n - 16 * t0];
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

template <int MT, int NC>
const void* int4_stream(int ng, bool zp) {
  constexpr int D = i4_depth(MT);
  if (zp)
    return ng == 4   ? (const void*)int4_stream_kernel<MT, NC, 4, true, D>
           : ng == 2 ? (const void*)int4_stream_kernel<MT, NC, 2, true, D>
                     : (const void*)int4_stream_kernel<MT, NC, 1, true, D>;
  return ng == 4   ? (const void*)int4_stream_kernel<MT, NC, 4, false, D>
         : ng == 2 ? (const void*)int4_stream_kernel<MT, NC, 2, false, D>
                   : (const void*)int4_stream_kernel<MT, NC, 1, false, D>;
}

// The wavefronts and their chunks (1, or 2 up to 16 rows) that take K in the
// fewest phases, counting two workgroups side by side on a compute unit as half;
// then the fewest phases, then the fewest idle chunk slots.
template <int MT>
hipError_t launch_int4_stream(Int4Args a, hipStream_t stream) {
  const int ng = a.group == 32 && a.K > 32 ? 4 : a.group == 64 && a.K > 64 ? 2 : 1;
  const int64_t nchunks = (a.K + kSt4Chunk - 1) / kSt4Chunk;
  // groups of a phase: at most its k / group, two more where they straddle
  auto pitch_of = [&](int64_t slots) { return std::min<int64_t>(a.groups, slots * kSt4Chunk / a.group + 2) | 1; };
  auto lds_of = [&](int64_t w, int64_t c) {
    return w * (i4_depth(MT) * c * kSt4Bytes + i4_buffers(MT) * 1024 * MT) + 128 * pitch_of(w * c);
  };
  int nc = 1, waves = 1;
  int64_t best = INT64_MAX;
  for (int c = 1; c <= (MT == 1 ? 2 : 1); ++c) {
    for (int64_t w = 1; w <= i4_max_waves(MT, c); ++w) {
      if (w > 1 && lds_of(w, c) > 152 * 1024) break;    // beside it the held sums of a few tiles
      const int64_t phases = (nchunks + w * c - 1) / (w * c);
      const int64_t side = std::max<int64_t>(1, std::min<int64_t>(2, i4_max_waves(MT, c) / w));
      const int64_t cost = phases * 1000000 / side + phases * 1000 + w * c;
      if (cost < best) {
        best = cost;
        nc = c;
        waves = (int)w;
      }
    }
  }
  const int64_t phases = (nchunks + waves * nc - 1) / (waves * nc);
  const int dev = current_device();
  const int64_t tiles = ((int64_t)a.N + 15) / 16;
  a.scale_pitch = (int)pitch_of((int64_t)waves * nc);
  int64_t lds = lds_of(waves, nc);
  const int per_cu = (int)std::max<int64_t>(
      1, std::min<int64_t>(phases > 1 ? std::min(2, i4_max_waves(MT, nc) / waves) : i4_max_waves(MT, nc) / waves, 158 * 1024 / (lds + (phases > 1 ? 8 * MT + 1 : 2) * 1024)));
  // a workgroup's tiles: their biases and, with several phases, their held sums fit beside
  const int64_t per_tile = 64 + (phases > 1 ? 1024 * MT : 0);
  const int64_t room = (158 * 1024 / per_cu - lds) / per_tile;
  const int64_t slots = (int64_t)device_cus(dev) * per_cu;
  const int64_t grid = std::min<int64_t>(tiles, slots * ((tiles + slots * room - 1) / (slots * room)));
  a.tiles_per_block = (int)((tiles + grid - 1) / grid);
  lds += a.tiles_per_block * per_tile;
  const void* fn = int4_stream<MT, 1>(ng, a.zeros != nullptr);
  if constexpr (MT == 1)
    if (nc == 2) fn = int4_stream<1, 2>(ng, a.zeros != nullptr);
  if (lds > 65536) {
    const hipError_t e = ensure_dynamic_lds(fn, dev, (int)lds);
    if (e != hipSuccess) return e;
  }
  const dim3 blocks((unsigned)grid, (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
  return launch_kernel_lds(fn, blocks, dim3(64 * waves), (size_t)lds, stream, a);
}

}  // namespace

namespace {

template <int MR, int SEG>
hipError_t launch_int4_dot(const Int4Args& a, hipStream_t stream) {
  const void* const fn = a.zeros ? (const void*)int4_dot_kernel<MR, SEG, true> : (const void*)int4_dot_kernel<MR, SEG, false>;
  const int dev = current_device();
  const int64_t blocks = ((int64_t)a.N + 15) / 16;
  const int64_t grid = std::min<int64_t>(blocks, (int64_t)device_cus(dev) * blocks_per_cu(fn, dev, 256, 0));
  return launch_kernel(fn, dim3((unsigned)grid), dim3(256), stream, a);
}

}  // namespace

// ---------------------------------------------------------------------------
// Enough weight rows, more than 16 activation rows or as the launcher says: a wavefront owns NT 16-row tiles
// for all of K, so its sums stay in its registers.  The eight wavefronts of a
// workgroup share x, 256 k a step in two LDS buffers, in the order that the MFMA
// reads it; the weights come through each wavefront's own ring of two chunks, its
// scales and zero points through its own piece of LDS.  x and scales are loaded
// three steps ahead into registers and stored one step ahead.  One barrier a
// step.  Where a group has 128 k or more, the sums of x that the offset needs fall
// out of the x stores.  The vector units bound it, LDS reads of x come next (half
// of either at 33 x 32000 x 4096 before the unpacking was cut from 11 to 7
// instructions a word): two tiles share each x fragment where the grid still fills the
// card.  33 x 32003 x 2080, groups of 32 with zero points: 24 to 27 us, 44 in the
// streamed form; 64 x 128256 x 4096: 106 us (2.6 TB/s, 640 TFLOP/s) against 165, one tile
// 145; 16 x 151936 x 5120 in groups of 32 with zero points 119 (3.8 TB/s) against 225.
// Beyond 64 rows every 64 read and unpack the weight again: 256 x 32000 x 4096 106 us
// (630 TFLOP/s), 2048 rows 820 us (650 TFLOP/s).
// ---------------------------------------------------------------------------
template <int MT, int NT, int NG, bool ZP>
__global__ __launch_bounds__(512) void int4_tile_kernel(Int4Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds8[];
  constexpr int D = 2;                                  // chunks of weights in flight; three are no faster
  constexpr int XB = MT * 8192;                         // bytes of an x buffer
  constexpr int COLS = 2 * NG, SP = COLS + 1;           // scales per row and step, and their LDS pitch
  constexpr int SI = (16 * NT * COLS + 63) / 64;        // scales per lane and step
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int K = a.K, N = a.N;
  const int64_t pitch = K >> 1;
  const int nch = (K + kSt4Chunk - 1) / kSt4Chunk;
  const int tiles = (N + 15) >> 4;
  const int mb = 16 * MT * blockIdx.y;
  uint8_t* const ring = lds8 + 2 * XB + wave * (D * NT * kSt4Bytes);
  float* const sums = reinterpret_cast<float*>(lds8 + 2 * XB + 8 * (D * NT * kSt4Bytes));   // [2][2][16 MT], NG == 1
  uint32_t* const scl = reinterpret_cast<uint32_t*>(sums + (NG == 1 ? 64 * MT : 0)) + wave * (16 * NT * SP);
  int tile[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) tile[t] = min(((int)blockIdx.x * 8 + wave) * NT + t, tiles - 1);   // a repeat is not stored

  // one base per tile and 32-bit offsets beside it
  uint32_t roff[NT][2];
  const uint8_t* wbase[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    wbase[t] = a.packed + (int64_t)16 * tile[t] * pitch;
#pragma unroll
    for (int j = 0; j < 2; ++j) roff[t][j] = (uint32_t)min(8 * j + (lane >> 3), N - 1 - 16 * tile[t]) * (uint32_t)pitch;
  }
  auto copy = [&](int c, int slot) {
    const uint32_t off = (uint32_t)st4_offset<int>(c, (int)pitch, lane);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      st4_copy_rows(wbase[t] + (roff[t][0] + off), wbase[t] + (roff[t][1] + off), ring + (slot * NT + t) * kSt4Bytes);
  };
  // scale e = lane + 64 i of a step: row e / COLS of the NT tiles, column e % COLS
  uint32_t sv[2][SI], zv[2][SI];
  // (2 c + col) / (128-k blocks per group), by a multiplication: exact to K = 2^22
  const uint32_t blocks = ((uint32_t)a.group + 127) / 128, per = (0x80000000u + blocks - 1) / blocks;
  auto scale_group = [&](int c, int col) {
    return NG == 1 ? (int)__umulhi(2u * (uint32_t)(2 * c + col), per) : COLS * c + col;
  };
  const int row0 = 16 * tile[0], last = N - 1 - row0;
  const uint8_t* const sbase = reinterpret_cast<const uint8_t*>(a.scales + (int64_t)row0 * a.groups);
  const uint8_t* const zbase = reinterpret_cast<const uint8_t*>(ZP ? a.zeros + (int64_t)(row0 >> 3) * a.groups : nullptr);
  uint32_t soff[SI], zoff[SI];
#pragma unroll
  for (int i = 0; i < SI; ++i) {
    const int row = min(min(lane + 64 * i, 16 * NT * COLS - 1) / COLS, last);
    soff[i] = (uint32_t)row * (uint32_t)a.groups;
    zoff[i] = (uint32_t)(row >> 3) * (uint32_t)a.groups;
  }
  auto load_scales = [&](int c, int set) {
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      const uint32_t j = (uint32_t)min(scale_group(c, min(lane + 64 * i, 16 * NT * COLS - 1) % COLS), a.groups - 1);
      sv[set][i] = *reinterpret_cast<const uint16_t*>(sbase + 2 * (soff[i] + j));
      if (ZP) zv[set][i] = *reinterpret_cast<const uint32_t*>(zbase + 4 * (zoff[i] + j));
    }
  };
  auto store_scales = [&](int c, int set) {
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      const int e = min(lane + 64 * i, 16 * NT * COLS - 1);
      uint32_t w = __float_as_uint(scale_value(sv[set][i], a.scale_f16));
      if (ZP) w |= (zv[set][i] >> (4 * (e / COLS & 7))) & 15u;
      if (scale_group(c, e % COLS) >= a.groups) w = 0;  // 0, lest an infinite scale meet x = 0
      scl[e / COLS * SP + e % COLS] = w;
    }
  };
  // x octet tid + 512 i of a step: row (tid + 512 i) / 32, k = 256 c + 8 ((tid + 512 i) % 32)
  u32x4 xv[2][MT];
  const int oct = tid & 31, o = oct & 15;
  const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(a.x + (int64_t)mb * K);
  uint32_t xoff[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xoff[i] = (uint32_t)min(16 * i + (tid >> 5), a.M - 1 - mb) * (uint32_t)K;
  auto load_x = [&](int c, int set) {
    const uint32_t k = (uint32_t)min(kSt4Chunk * c + 8 * oct, K - 8);
#pragma unroll
    for (int i = 0; i < MT; ++i) xv[set][i] = *reinterpret_cast<const u32x4*>(xbase + 2 * (xoff[i] + k));
  };
  // MFMA step s, lane quarter g of octet o of a 128-k half; the slot is swizzled
  // by o so that 16 octets of a row spread over the banks
  const int xw = ((oct >> 4) * 4 + (NG == 1 ? o & 3 : o >> 2)) * 1024 + ((NG == 1 ? o >> 2 : o & 3) * 16 + ((tid >> 5) ^ o)) * 16;
  auto store_x = [&](int c, int set) {
    uint8_t* const b = lds8 + (c & 1) * XB + xw;
    const bool in = kSt4Chunk * c + 8 * oct < K;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const u32x4 v = in ? xv[set][i] : u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<bf16x8*>(b + i * 8192) = reorder_x(v);
      if (NG == 1) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = v[e];
          s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, 0x3F803F80u), s, false);
        }
        s = dpp_row_sum(s);
        if (o == 0) sums[((c & 1) * 2 + (oct >> 4)) * 16 * MT + 16 * i + (tid >> 5)] = s;
      }
    }
  };

  load_x(0, 0);
  load_scales(0, 0);
  __asm__ volatile("" ::: "memory");
  load_x(min(1, nch - 1), 1);
  load_scales(min(1, nch - 1), 1);
  __asm__ volatile("" ::: "memory");
  copy(0, 0);
  __asm__ volatile("" ::: "memory");
  store_x(0, 0);
  store_scales(0, 0);
  load_x(min(2, nch - 1), 0);
  load_scales(min(2, nch - 1), 0);
  __asm__ volatile("" ::: "memory");
  copy(min(1, nch - 1), 1);
  __asm__ volatile("" ::: "memory");

  f32x4 total[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < MT; ++i) total[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  int xr[4];                                            // the lane's slot in step s's 64
#pragma unroll
  for (int s = 0; s < 4; ++s) xr[s] = s * 1024 + (g * 16 + (r ^ (NG == 1 ? 4 * g + s : 4 * s + g))) * 16;

  int slot = 0;
  auto step = [&](int c, int set) {                     // set: (c + 1) % 2
    st4_barrier();
    // chunk c's copies, and the x and scales of c + 1: one step's loads and copies are younger
    __builtin_amdgcn_s_waitcnt(st4_vm(2 * NT + MT + SI * (ZP ? 2 : 1)));
    __builtin_amdgcn_sched_barrier(0);                  // no use of those moves above the wait
    __asm__ volatile("" ::: "memory");
    u32x4 w[NT][2];
    uint32_t sw[NT][COLS];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) w[t][h] = st4_read(ring + (slot * NT + t) * kSt4Bytes, r, 4 * h + g);
#pragma unroll
      for (int j = 0; j < COLS; ++j) sw[t][j] = scl[(16 * t + r) * SP + j];
    }
    __builtin_amdgcn_s_waitcnt(kSt4Lgkm0);              // the region may now be refilled
    __asm__ volatile("" ::: "memory");
    store_x(c + 1, set);
    store_scales(c + 1, set);
    load_x(min(c + 3, nch - 1), set);
    load_scales(min(c + 3, nch - 1), set);
    __asm__ volatile("" ::: "memory");
    copy(min(c + D, nch - 1), slot);
    __asm__ volatile("" ::: "memory");                  // issued now, not at the step's end
    slot ^= 1;

    const uint8_t* const xb = lds8 + (c & 1) * XB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 acc[NT][MT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (NG > 1) transpose4(w[t][h]);
      if (NG == 1) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const f32x4 sx = *reinterpret_cast<const f32x4*>(sums + ((c & 1) * 2 + h) * 16 * MT + 16 * i + 4 * g);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float off = ZP ? -16.0f - (float)(sw[t][h] & 15u) : -24.0f;
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[t][i][v] = off * sx[v];
          }
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        constexpr int kSteps = 4 / NG;                  // MFMA steps per group
        const bool fresh = NG > 1 && s % kSteps == 0;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        bf16x8 xa[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) xa[i] = *reinterpret_cast<const bf16x8*>(xb + i * 8192 + h * 4096 + xr[s]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t sb = sw[t][h * NG + s / kSteps];
          const bf16x8 wb = codes_bf16(w[t][h][s]);
          const uint32_t ob = ZP ? (0xC180u | (sb & 15u) << 3) * 0x10001u : 0xC1C0C1C0u;
          const u32x4 obits = {ob, ob, ob, ob};
          const bf16x8 off = __builtin_bit_cast(bf16x8, obits);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            acc[t][i] = mfma_i4(xa[i], wb, fresh ? zero : acc[t][i]);
            if (NG > 1) acc[t][i] = mfma_i4(xa[i], off, acc[t][i]);
          }
          if (s % kSteps == kSteps - 1) {
            const float sc = __uint_as_float(ZP ? sb & ~15u : sb);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int v = 0; v < 4; ++v) total[t][i][v] = __builtin_fmaf(sc, acc[t][i][v], total[t][i][v]);
          }
        }
      }
    }
  };
  // whole pairs of steps: a step past K adds 0, and one block keeps the compiler's waits out
  for (int c = 0; c < nch; c += 2) {
    step(c, 1);
    step(c + 1, 0);
  }
  __builtin_amdgcn_s_waitcnt(st4_vm(0));                // trailing copies land before the LDS is given up
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = 16 * (((int)blockIdx.x * 8 + wave) * NT + t) + r;
    if (n >= N) continue;
    const float bias = a.bias ? __uint_as_float((uint32_t)a.bias[n] << 16) : 0.0f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int m = mb + 16 * i + 4 * g + v;
        if (m < a.M) a.y[(int64_t)m * N + n] = __builtin_bit_cast(uint16_t, (__bf16)(total[t][i][v] + bias));
      }
  }
}

namespace {

template <int MT, int NT>
hipError_t launch_int4_tiles(const Int4Args& a, const dim3& blocks, hipStream_t stream) {
  const int ng = a.group == 32 && a.K > 32 ? 4 : a.group == 64 && a.K > 64 ? 2 : 1;
  const void* fn;
  if (a.zeros)
    fn = ng == 4   ? (const void*)int4_tile_kernel<MT, NT, 4, true>
         : ng == 2 ? (const void*)int4_tile_kernel<MT, NT, 2, true>
                   : (const void*)int4_tile_kernel<MT, NT, 1, true>;
  else
    fn = ng == 4   ? (const void*)int4_tile_kernel<MT, NT, 4, false>
         : ng == 2 ? (const void*)int4_tile_kernel<MT, NT, 2, false>
                   : (const void*)int4_tile_kernel<MT, NT, 1, false>;
  const int lds = 2 * MT * 8192 + 8 * 2 * NT * kSt4Bytes + (ng == 1 ? 256 * MT : 0) + 8 * 64 * NT * (2 * ng + 1);
  if (lds > 65536) {
    const hipError_t e = ensure_dynamic_lds(fn, current_device(), lds);
    if (e != hipSuccess) return e;
  }
  return launch_kernel_lds(fn, blocks, dim3(512), (size_t)lds, stream, a);
}

// Two tiles a wavefront where that takes fewer rounds of workgroups, a round
// counted 1.6 times as long (64 x 128256 x 4096: 53 and 36 us a round; 1.1 to 1.5
// times where one round is all, so that one tile is right there).  Over 17 to 160
// rows, N of 4000 to 128256 and K of 2048 to 8192 it takes the faster one within 6 %.
template <int MT>
hipError_t launch_int4_tile(const Int4Args& a, hipStream_t stream) {
  const int64_t cus = device_cus(current_device());
  const int64_t mblocks = ((int64_t)a.M + 16 * MT - 1) / (16 * MT);
  const int64_t one = ((int64_t)a.N + 127) / 128, two = ((int64_t)a.N + 255) / 256;
  const int64_t rounds1 = (one * mblocks + cus - 1) / cus, rounds2 = (two * mblocks + cus - 1) / cus;
  if (8 * rounds2 < 5 * rounds1) return launch_int4_tiles<MT, 2>(a, dim3((unsigned)two, (unsigned)mblocks), stream);
  return launch_int4_tiles<MT, 1>(a, dim3((unsigned)one, (unsigned)mblocks), stream);
}

}  // namespace

hipError_t launch_int4_gemm(Int4Args a, hipStream_t stream) {
  // One or two rows whose x fits in the lanes' registers (K to 8192, and 2048).
  // The dot kernel against the streamed one, M = 1: 151936 x 5120 82 and 84 us,
  // 128256 x 6656 100 and 131, 128256 x 1280 in groups of 32 23 and 38, 1024 x 1280 3.6
  // and 5.6; M = 2, 128256 x 2048: 33.4 and 32.8, beyond that K 128256 x 4096 75 and 53.
  const int64_t seg = ((int64_t)a.K + 2047) / 2048;
  if (a.M == 1 && seg == 1) return launch_int4_dot<1, 1>(a, stream);
  if (a.M == 1 && seg == 2) return launch_int4_dot<1, 2>(a, stream);
  if (a.M == 1 && seg == 3) return launch_int4_dot<1, 3>(a, stream);
  if (a.M == 1 && seg == 4) return launch_int4_dot<1, 4>(a, stream);
  if (a.M == 2 && seg == 1) return launch_int4_dot<2, 1>(a, stream);
  // The tile kernel where one tile a wavefront gives two fifths of the compute
  // units a workgroup (64 x 12000 x 8192: 61 us, streamed 60; 33 x 16000 x 4096 26 and
  // 27; 64 x 4096 x 4096 38 and 23; 16 x 13000 x 2048 9 and 13, x 8192 27 and 30), and K
  // leaves its 32-bit offsets in range.  Up to 16 rows in groups of 128 or more the
  // streamed form, whose work divides evenly, keeps the sizes that would leave a
  // second or later round of workgroups (two a compute unit) less than three quarters
  // full, if K is 16 to 20 chunks, one phase of eight to ten wavefronts.  Streamed and
  // tiles, N = 70000, 98304, 140000 at K = 5120: 3 rows 45 57 78, 51 56 86 us; 16 rows 48 62
  // 85, 59 66 102; at 4096: 35 44 60, 36 41 63; 37 49 63, 41 47 73.  At other K it
  // loses: 2560 16 rows 37 46 60, 28 32 49; 6144 62 98 120, 65 74 113; 8192 about even.
  const int64_t cus = device_cus(current_device());
  const int64_t nblocks = ((int64_t)a.N + 127) / 128, mblocks = a.M <= 48 ? 1 : ((int64_t)a.M + 63) / 64;
  if (5 * nblocks * mblocks >= 2 * cus && a.K <= 1 << 22) {
    const int64_t over = nblocks % (2 * cus);
    const int64_t nchunks = ((int64_t)a.K + kSt4Chunk - 1) / kSt4Chunk;
    const bool uneven = nblocks > 2 * cus && over != 0 && 2 * over < 3 * cus && nchunks >= 16 && nchunks <= 20;
    const bool small_groups = a.group < 128 && a.K > a.group;
    if (a.M <= 16 && (small_groups || !uneven)) return launch_int4_tiles<1, 1>(a, dim3((unsigned)nblocks), stream);
    if (a.M > 16 && a.M <= 32) return launch_int4_tile<2>(a, stream);
    if (a.M > 32 && a.M <= 48) return launch_int4_tile<3>(a, stream);
    if (a.M > 48) return launch_int4_tile<4>(a, stream);
  }
  if (a.M <= 16) return launch_int4_stream<1>(a, stream);
  if (a.M <= 32) return launch_int4_stream<2>(a, stream);
  if (a.M <= 48) return launch_int4_stream<3>(a, stream);
  return launch_int4_stream<4>(a, stream);
}

}  // namespace nvfp4
