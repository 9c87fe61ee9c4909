// The whole W4A16 NVFP4 expert layer for a few tokens (T <= 16), from the
// router's logits, in two kernels (gfx950).
//
// Weights as in nvfp4_moe.hip (vLLM modelopt.py, ModelOptNvFp4FusedMoE,
// use_a16).  For token t the router's scores are softmax or sigmoid of its
// logits, the topk largest logits (of score + bias, with a bias) are chosen,
// equal ones by the lower index, and
//   out[t] = sum_j w[t, j] W2_e (silu(W1_e x[t]) * (W3_e x[t])),  e = ids[t, j].
//
// Up kernels: every workgroup routes all tokens by itself (a few hundred
// logits, one wavefront per token; cheaper than a launch), lists the chosen
// experts in order and walks its share of (expert, 16 columns of I), gate and up
// rows of the same columns together, so the activation is applied at once.
// Down kernels: K = I of all chosen experts, each expert's sum weighted by w[t, j].
// The MFMA's columns are the tokens themselves (16 at most), a token that did
// not choose the expert is a column of zeros: no gathering, no lists of pairs.
//
// HBM bounds both: 0.5625 bytes per weight of the chosen experts.  The streamed form
// (further down) serves H and I that are multiples of 32, from 64.  8 experts, 4096 x
// 14336, top-2: T = 1 49 us (198 MB, 4.0 TB/s: 28 us up, 22 us down), T = 16 163 us
// (785 MB, 4.8 TB/s); 64 experts of 2048 x 1024, T = 4 36 us.  The register form here
// serves the other sizes (at T = 1, 16 of the first layer it took 65 and 211 us; 8
// experts of 4112 x 14336 102 and 421 us).  H beyond 4096 takes the up kernel several
// passes, whose sums wait in LDS: 8 of 64 experts of 7168 x 2048, T = 8 288 us (3.6 TB/s).
//
// Register form.  A workgroup of the down kernel owns 16 output columns, its
// wavefronts split the K of all chosen experts, nothing per pair is written.
// Weights stream straight to registers, one 256-k chunk ahead: lane (r, g) =
// (lane % 16, lane / 16) holds row r's codes of k = 256 c + 64 g + [0, 64) (two
// 16-byte loads) and their four block scales (one 4-byte load); MFMA step s
// multiplies k = 64 g + 8 s + [0, 8) of each g.  A code times its block scale is
// exact in bf16.  The hidden activation is kept as a bf16 pair hi + lo (16 bits
// of it, twice the output's; a third part, float32's 24 bits, takes T = 1 at 4112 x
// 14336 from 102 to 120 us), so that the only rounding to bf16 is the output's.
#include <algorithm>

#include "nvfp4_device.hpp"
#include "nvfp4_launch.hpp"
#include "stream4.hpp"

namespace nvfp4 {

namespace {

constexpr int kMdWaves = 4;                  // up kernel
constexpr int kMdDownWaves = 8;
constexpr int kMdChunk = 256;
constexpr int kMdMaxPairs = kMoeDecodeMaxT * kMoeDecodeMaxTopk;

struct __attribute__((packed, aligned(8))) Vec16A8 { u32x4 v; };
struct __attribute__((packed, aligned(1))) Word4A1 { uint32_t v; };

__device__ __forceinline__ f32x4 mfma_md(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Maximum over the wavefront, in every lane.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true)));
  auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_row_sum(v);
  auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Routing of token t by one wavefront; expert e = lane + 64 i.  A logit of -inf
// or NaN is never chosen; slots without an expert get id -1, weight 0.
template <int NI>
__device__ __forceinline__ void route_token(const MoeDecodeArgs& a, int t, int lane, int32_t* ids, float* weights) {
  float logit[NI], score[NI], sel[NI];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    float l = -INFINITY;
    if (e < a.E) {
      const int64_t at = (int64_t)t * a.E + e;
      l = a.router_f32 ? static_cast<const float*>(a.router)[at]
                       : __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.router)[at] << 16);
    }
    logit[i] = l > -INFINITY ? l : -INFINITY;
    top = fmaxf(top, logit[i]);
  }
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NI; ++i) score[i] = 1.0f / (1.0f + expf(-logit[i]));
  } else {
    top = wave_max(top);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      score[i] = logit[i] > -INFINITY ? expf(logit[i] - top) : 0.0f;
      sum += score[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < NI; ++i) score[i] = score[i] / sum;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 64 * i;
    sel[i] = logit[i];
    if (a.bias && logit[i] > -INFINITY) {
      const float b = score[i] + a.bias[e];
      sel[i] = b > -INFINITY ? b : -INFINITY;
    }
  }
  float mine = 0.0f, total = 0.0f;                     // lane j keeps slot j
  int my_id = -1;
  for (int j = 0; j < a.topk; ++j) {
    float best = sel[0];
#pragma unroll
    for (int i = 1; i < NI; ++i) best = fmaxf(best, sel[i]);
    best = wave_max(best);
    if (best == -INFINITY) break;
    bool found = false;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint64_t hit = __ballot(sel[i] == best);
      if (!found && hit != 0) {
        found = true;
        const int src = __ffsll((unsigned long long)hit) - 1;
        const float w = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(score[i]), src));
        if (lane == src) sel[i] = -INFINITY;
        if (lane == j) {
          mine = w;
          my_id = src + 64 * i;
        }
        total += w;
      }
    }
    if (!found) break;                                  // only a NaN score gets here
  }
  if (a.renormalize && total > 0.0f) mine /= total;
  if (lane < a.topk) {
    ids[t * a.topk + lane] = my_id;
    weights[t * a.topk + lane] = mine * a.weight_scale;
  }
}

// A 256-k chunk of one weight row, as lane (r, g) holds it.
struct Codes {
  u32x4 w[2];
  uint32_t s;
};

__device__ __forceinline__ void load_codes(const uint8_t* row, const uint8_t* srow, int c, int g, int K, Codes* o) {
  const int k0 = kMdChunk * c + 64 * g;
  if (kMdChunk * (c + 1) <= K) {                        // uniform over the wavefront
    o->w[0] = reinterpret_cast<const Vec16A8*>(row + (k0 >> 1))->v;
    o->w[1] = reinterpret_cast<const Vec16A8*>(row + (k0 >> 1) + 16)->v;
    o->s = reinterpret_cast<const Word4A1*>(srow + (k0 >> 4))->v;
    return;
  }
  o->s = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = k0 + 32 * h;
    u32x4 w = {0u, 0u, 0u, 0u};
    if (k + 32 <= K) {
      w = reinterpret_cast<const Vec16A8*>(row + (k >> 1))->v;
    } else if (k < K) {                                 // K % 32 == 16
      const uint2 v = *reinterpret_cast<const uint2*>(row + (k >> 1));
      w[0] = v.x;
      w[1] = v.y;
    }
    o->w[h] = w;
  }
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (k0 + 16 * b < K) o->s |= (uint32_t)srow[(k0 >> 4) + b] << (8 * b);
}

template <int S>
__device__ __forceinline__ bf16x8 step_weight(const Codes& q) {
  return dequant8(q.w[S >> 2][S & 3], NVFP4_E4M3_TO_F32(q.s, S >> 1));
}

// Activation fragments of chunk c: row + 256 c + 64 g + 8 s, 0 beyond K or where
// the lane's column has none.
__device__ __forceinline__ void load_x(const uint16_t* row, bool use, int c, int g, int K, u32x4* xv) {
  const int k0 = kMdChunk * c + 64 * g;
#pragma unroll
  for (int s = 0; s < 8; ++s)
    xv[s] = use && k0 + 8 * s < K ? *reinterpret_cast<const u32x4*>(row + k0 + 8 * s) : u32x4{0u, 0u, 0u, 0u};
}

// Routes every token of the batch and lists the chosen experts in increasing
// order, in LDS (one workgroup of W wavefronts); workgroup 0 leaves the results
// for the second kernel and the caller.  flag has 64 NI words.
template <int NI>
__device__ __forceinline__ int route_all(const MoeDecodeArgs& a, int32_t* ids, float* weights, int32_t* flag,
                                         int32_t* list, int32_t* n_active) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int threads = blockDim.x, pairs = a.T * a.topk;
  for (int e = tid; e < 64 * NI; e += threads) flag[e] = 0;
  for (int t = wave; t < a.T; t += threads >> 6) route_token<NI>(a, t, lane, ids, weights);
  __syncthreads();
  for (int p = tid; p < pairs; p += threads)
    if (ids[p] >= 0) flag[ids[p]] = 1;
  __syncthreads();
  if (wave == 0) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool on = flag[64 * i + lane] != 0;
      const uint64_t all = __ballot(on);
      if (on) list[n + __popcll(all & (((uint64_t)1 << lane) - 1))] = 64 * i + lane;
      n += __popcll(all);
    }
    if (lane == 0) *n_active = n;
  }
  __syncthreads();
  const int active = *n_active;
  if (blockIdx.x == 0) {
    for (int p = tid; p < pairs; p += threads) {
      a.ids[p] = ids[p];
      a.weights[p] = weights[p];
      if (a.ids_out) a.ids_out[p] = ids[p];
      if (a.weights_out) a.weights_out[p] = weights[p];
    }
    for (int s = tid; s < active; s += threads) a.list[s] = list[s];
    if (tid == 0) *a.active = active;
    for (int i = tid; i < a.n_counters; i += threads) a.counters[i] = 0;
  }
  return active;
}

#define NVFP4_MD_STEPS(F) F(0) F(1) F(2) F(3) F(4) F(5) F(6) F(7)

}  // namespace

template <int NI>
__global__ __launch_bounds__(64 * kMdWaves) void moe_decode_up_kernel(MoeDecodeArgs a) {
  __shared__ int32_t sh_ids[kMdMaxPairs];
  __shared__ float sh_w[kMdMaxPairs];
  __shared__ int32_t sh_flag[64 * NI];
  __shared__ int32_t sh_list[kMdMaxPairs];
  __shared__ int32_t sh_active;
  __shared__ float red[kMdWaves][8][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int active = route_all<NI>(a, sh_ids, sh_w, sh_flag, sh_list, &sh_active);

  const int splitk = a.splitk, rg = wave / splitk, ph = wave - rg * splitk;
  const int per = kMdWaves / splitk;                    // 16-column tiles per workgroup and item
  const int tiles = a.I >> 4, groups = (tiles + per - 1) / per;
  const int K = a.H, nch = (K + kMdChunk - 1) / kMdChunk;
  const int64_t prow = K >> 1, srow = K >> 4;
  for (int item = blockIdx.x; item < active * groups; item += gridDim.x) {
    const int slot = item / groups, e = sh_list[slot];
    const int tile = (item - slot * groups) * per + rg;
    const bool live = tile < tiles;
    const int64_t gate = (int64_t)e * 2 * a.I + 16 * min(tile, tiles - 1) + r, up = gate + a.I;
    const uint8_t* const gp = a.w13_packed + gate * prow;
    const uint8_t* const gs = a.w13_scales + gate * srow;
    const uint8_t* const upp = a.w13_packed + up * prow;
    const uint8_t* const ups = a.w13_scales + up * srow;
    int pair = -1;                                      // of this lane's token with expert e
    if (r < a.T)
      for (int j = 0; j < a.topk; ++j)
        if (sh_ids[r * a.topk + j] == e) pair = r * a.topk + j;
    const uint16_t* const xr = a.x + (int64_t)min(r, a.T - 1) * K;

    f32x4 accg = {0.f, 0.f, 0.f, 0.f}, accu = {0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int c, const Codes& qg, const Codes& qu) {
      u32x4 xv[8];
      load_x(xr, pair >= 0, c, g, K, xv);
#define NVFP4_MD_UP(S)                                         \
  {                                                            \
    const bf16x8 b = __builtin_bit_cast(bf16x8, xv[S]);        \
    accg = mfma_md(step_weight<S>(qg), b, accg);               \
    accu = mfma_md(step_weight<S>(qu), b, accu);               \
  }
      NVFP4_MD_STEPS(NVFP4_MD_UP)
#undef NVFP4_MD_UP
    };
    if (live) {
      Codes g0, u0, g1, u1;
      if (ph < nch) {
        load_codes(gp, gs, ph, g, K, &g0);
        load_codes(upp, ups, ph, g, K, &u0);
      }
      for (int c = ph; c < nch; c += 2 * splitk) {
        if (c + splitk < nch) {
          load_codes(gp, gs, c + splitk, g, K, &g1);
          load_codes(upp, ups, c + splitk, g, K, &u1);
        }
        compute(c, g0, u0);
        if (c + splitk >= nch) break;
        if (c + 2 * splitk < nch) {
          load_codes(gp, gs, c + 2 * splitk, g, K, &g0);
          load_codes(upp, ups, c + 2 * splitk, g, K, &u0);
        }
        compute(c + splitk, g1, u1);
      }
    }
    if (splitk > 1) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        red[wave][v][lane] = accg[v];
        red[wave][4 + v][lane] = accu[v];
      }
      __syncthreads();
      if (ph == 0) {
        for (int q = 1; q < splitk; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            accg[v] += red[wave + q][v][lane];
            accu[v] += red[wave + q][4 + v][lane];
          }
      }
      __syncthreads();                                  // red is written again by the next item
    }
    if (live && ph == 0 && pair >= 0) {
      const float gsc = a.w13_gs[e];
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float gv = accg[v] * gsc, uv = accu[v] * gsc;
        const float act = gv / (1.0f + expf(-gv)) * uv;
        hi[v] = __builtin_bit_cast(uint16_t, (__bf16)act);
        const float rest = act - __uint_as_float(hi[v] << 16);
        // an infinite activation has no rest
        lo[v] = __builtin_bit_cast(uint16_t, (__bf16)(fabsf(act) < INFINITY ? rest : 0.0f));
      }
      const int64_t at = (int64_t)pair * a.I + 16 * tile + 4 * g;
      *reinterpret_cast<uint2*>(a.a_hi + at) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
      *reinterpret_cast<uint2*>(a.a_lo + at) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
    }
  }
}

__global__ __launch_bounds__(64 * kMdDownWaves) void moe_decode_down_kernel(MoeDecodeArgs a) {
  __shared__ float red[kMdDownWaves][4][64];
  __shared__ int sh_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x / a.down_split, part = blockIdx.x - tile * a.down_split;
  const int K = a.I, nch = (K + kMdChunk - 1) / kMdChunk;
  const int64_t prow = K >> 1, srow = K >> 4;
  const int active = *a.active;
  // this wavefront's run of the (expert, chunk) units
  const int units = active * nch, workers = a.down_split * kMdDownWaves;
  const int me = part * kMdDownWaves + wave;
  const int u0 = (int)((int64_t)units * me / workers), u1 = (int)((int64_t)units * (me + 1) / workers);

  f32x4 total = {0.f, 0.f, 0.f, 0.f};
  int u = u0;
  while (u < u1) {
    const int slot = u / nch, e = __builtin_amdgcn_readfirstlane(a.list[slot]);
    const int c0 = u - slot * nch, c1 = min(nch, c0 + u1 - u);
    u += c1 - c0;
    int pair = -1;
    float w = 0.0f;
    if (r < a.T)
      for (int j = 0; j < a.topk; ++j)
        if (a.ids[r * a.topk + j] == e) {
          pair = r * a.topk + j;
          w = a.weights[pair];
        }
    const int64_t row = (int64_t)e * a.H + 16 * tile + r;
    const uint8_t* const wp = a.w2_packed + row * prow;
    const uint8_t* const ws = a.w2_scales + row * srow;
    const uint16_t* const hi = a.a_hi + (int64_t)max(pair, 0) * K;
    const uint16_t* const lo = a.a_lo + (int64_t)max(pair, 0) * K;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int c, const Codes& q) {
      u32x4 xh[8], xl[8];
      load_x(hi, pair >= 0, c, g, K, xh);
      load_x(lo, pair >= 0, c, g, K, xl);
#define NVFP4_MD_DOWN(S)                                            \
  {                                                                 \
    const bf16x8 wb = step_weight<S>(q);                            \
    acc = mfma_md(wb, __builtin_bit_cast(bf16x8, xl[S]), acc);      \
    acc = mfma_md(wb, __builtin_bit_cast(bf16x8, xh[S]), acc);      \
  }
      NVFP4_MD_STEPS(NVFP4_MD_DOWN)
#undef NVFP4_MD_DOWN
    };
    Codes q0, q1;
    load_codes(wp, ws, c0, g, K, &q0);
    for (int c = c0; c < c1; c += 2) {
      if (c + 1 < c1) load_codes(wp, ws, c + 1, g, K, &q1);
      compute(c, q0);
      if (c + 1 >= c1) break;
      if (c + 2 < c1) load_codes(wp, ws, c + 2, g, K, &q0);
      compute(c + 1, q1);
    }
    if (pair >= 0) {
      const float f = w * a.w2_gs[e];
#pragma unroll
      for (int v = 0; v < 4; ++v) total[v] = __builtin_fmaf(f, acc[v], total[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave][v][lane] = total[v];
  __syncthreads();
  // thread (t, n): row n = 4 g + v of the tile, token t
  const int t = tid >> 4, n = tid & 15;
  float sum = 0.0f;
  const bool mine = t < a.T;
  if (mine)
#pragma unroll
    for (int q = 0; q < kMdDownWaves; ++q) sum += red[q][n & 3][16 * (n >> 2) + t];
  if (a.down_split > 1) {
    // the workgroup that arrives last adds the parts in order: the result does
    // not depend on which one that is
    float* const parts = a.parts + (int64_t)tile * a.down_split * 256;
    if (mine) __hip_atomic_store(parts + part * 256 + tid, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __threadfence();
    __syncthreads();
    if (tid == 0)
      sh_last = __hip_atomic_fetch_add(a.counters + tile, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (sh_last != a.down_split - 1) return;
    __threadfence();
    sum = 0.0f;
    if (mine)
      for (int q = 0; q < a.down_split; ++q)
        sum += __hip_atomic_load(parts + q * 256 + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (mine) a.out[(int64_t)t * a.H + 16 * tile + n] = __builtin_bit_cast(uint16_t, (__bf16)sum);
}

// ---------------------------------------------------------------------------
// The streamed form (H and I multiples of 32, from 64; stream4.hpp's scheme).
//
// A wavefront keeps the activations of its chunks as f16 MFMA operands, scaled by a power
// of two of its own per token, chosen so that the largest magnitude among its
// k lands in [2^14, 2^15): a bf16 value down to 2^-28 of that largest one stays
// exact; a float32 one (the hidden activation, which is stored as float32) takes two
// operands, its first 11 bits and the next, which HBM hides (T = 16, 8 experts of 4096 x
// 14336: 164 us, 167 with the first operand alone and the loop as it was; 64 experts of
// 2048 x 1024 36.3 and 35.1).  Their registers leave none to spare: the activations are
// loaded once for each run of tiles, not inside its steps, and addresses are 32-bit
// offsets.  The wavefront's sums are scaled back
// before they meet the others', so the scales need not agree.  In f16 a code
// times its block scale costs half of what it costs in bf16 (and is as exact).
// ---------------------------------------------------------------------------
namespace {

__device__ __forceinline__ f32x4 mfma_md16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Largest of the four lanes of a column (r, r + 16, r + 32, r + 48).
__device__ __forceinline__ uint32_t column_max(uint32_t v) {
  auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(p[0], p[1]);
  p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(p[0], p[1]);
}

// Exponent p with the magnitude (float32 bits) times 2^-p in [2^14, 2^15).
__device__ __forceinline__ int scale_exponent(uint32_t mag) {
  return mag < 0x00800000u ? 0 : max(-126, (int)(mag >> 23) - 141);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ f16x8 pack_f16(const float* v, float down) {
  f16x8 h;
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = (_Float16)(v[e] * down);
  return h;
}

// The same as two parts of 11 bits each, the first cut (one conversion for two
// values) and the second what that left, cut too: 20 bits at least.  What an infinite
// value leaves is NaN; the minimum, which no finite rest (below 16) reaches, makes it a
// number.
__device__ __forceinline__ f16x8 pack_f16_pair(const float* v, float down, f16x8* rest) {
  f16x8 h;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const auto hi = __builtin_amdgcn_cvt_pkrtz(v[e] * down, v[e + 1] * down);
    h[e] = (_Float16)hi[0];
    h[e + 1] = (_Float16)hi[1];
    const auto lo = __builtin_amdgcn_cvt_pkrtz(fminf(__builtin_fmaf(v[e], down, -(float)h[e]), 16.0f),
                                               fminf(__builtin_fmaf(v[e + 1], down, -(float)h[e + 1]), 16.0f));
    (*rest)[e] = (_Float16)lo[0];
    (*rest)[e + 1] = (_Float16)lo[1];
  }
  return h;
}

// Block scales of rows for the workgroup: thread `it` holds word it % words of row
// it / words of a 16-row tile; nb = bytes of a row's scales.
__device__ __forceinline__ int scale_word_offset(int word, int nb) { return min(4 * word, nb - 4); }
__device__ __forceinline__ uint32_t scale_word(uint32_t loaded, int word, int nb) {
  const int shift = 8 * (4 * word - scale_word_offset(word, nb));
  return shift < 32 ? loaded >> shift : 0u;              // blocks past the row's end have scale 0
}
__device__ __forceinline__ uint32_t load_scale_word(const uint8_t* row, int word, int nb) {
  return scale_word(reinterpret_cast<const Word4A1*>(row + scale_word_offset(word, nb))->v, word, nb);
}

struct ScaleSplit {
  float s[4];
  f16x2 mu[4];
};
__device__ __forceinline__ ScaleSplit split4(uint32_t w) {
  ScaleSplit o;
  o.s[0] = NVFP4_E4M3_TO_F32(w, 0);
  o.s[1] = NVFP4_E4M3_TO_F32(w, 1);
  o.s[2] = NVFP4_E4M3_TO_F32(w, 2);
  o.s[3] = NVFP4_E4M3_TO_F32(w, 3);
#pragma unroll
  for (int b = 0; b < 4; ++b) o.mu[b] = scale_mantissa_f16(o.s[b]);
  return o;
}

// acc += (tile chunk) x (activations of the chunk, with their rests where PAIR),
// k = 64 g + 8 s + [0, 8).
template <bool PAIR>
__device__ __forceinline__ f32x4 chunk_product(u32x4 w0, u32x4 w1, uint32_t sw, const f16x8* xb, const f16x8* rest,
                                               f32x4 acc) {
  const ScaleSplit q = split4(sw);
  f32x4 odd = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const uint32_t w = s < 4 ? w0[s & 3] : w1[s & 3];
    const f16x8 a = dequant8_f16(w, q.s[s >> 1], q.mu[s >> 1]);
    if (PAIR && (s & 1)) odd = mfma_md16(a, rest[s], odd);
    if (PAIR && !(s & 1)) acc = mfma_md16(a, rest[s], acc);
    if (s & 1)
      odd = mfma_md16(a, xb[s], odd);
    else
      acc = mfma_md16(a, xb[s], acc);
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] += odd[v];
  return acc;
}

constexpr int kMdDepth = 2;                  // tiles in flight per wavefront

// Floats between two rows of the hidden activation: whole chunks.
__device__ __host__ constexpr int64_t act_pitch(int64_t I) { return (I + kSt4Chunk - 1) / kSt4Chunk * kSt4Chunk; }

// LDS words of a row's scales for W wavefronts of NC chunks, padded to spread the rows.
__device__ __host__ constexpr int md_scale_pitch(int slots) { return 4 * slots + 1; }

}  // namespace

// Up: a[pair, i] = silu(gate) * up, float32.  Units (expert, 16 columns of I) are
// dealt to the workgroups in contiguous runs; each is two tiles, the gate's and
// the up's.
template <int NI, int NC, bool PASSES>
__global__ __launch_bounds__(1024) void moe_stream_up_kernel(MoeDecodeArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds8[];
  __shared__ int32_t sh_ids[kMdMaxPairs];
  __shared__ float sh_w[kMdMaxPairs];
  __shared__ int32_t sh_flag[64 * NI];
  __shared__ int32_t sh_list[kMdMaxPairs];
  __shared__ int32_t sh_active;
  __shared__ float sh_gs[kMdMaxPairs];                    // of the chosen experts: no load in the loop but the stream's
  constexpr int D = kMdDepth;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int W = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int K = a.H, nb = K >> 4, nch = (K + kSt4Chunk - 1) / kSt4Chunk;
  const int64_t pitch = K >> 1;
  const int phases = PASSES ? (nch + W * NC - 1) / (W * NC) : 1;
  uint8_t* const ring = lds8 + wave * (D * NC * kSt4Bytes);
  float* const red = reinterpret_cast<float*>(lds8 + W * (D * NC * kSt4Bytes));          // [W][2][256]
  const int spitch = md_scale_pitch(W * NC);
  uint32_t* const scl = reinterpret_cast<uint32_t*>(red + W * 512);                      // [2][16][spitch]
  float* const held = reinterpret_cast<float*>(scl + 32 * spitch);                       // [units][512], several phases

  // activations of the wavefront's chunks: column r is token r (the first ones
  // before the routing, whose latency covers theirs)
  f16x8 xb[NC][8];
  float back;
  auto load_tokens = [&](int c0) {
    u32x4 xv[NC][8];
    uint32_t mag = 0;
    const uint16_t* const xrow = a.x + (int64_t)min(r, a.T - 1) * K;
#pragma unroll
    for (int q = 0; q < NC; ++q) {
      load_x(xrow, true, c0 + q, g, K, xv[q]);
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) mag = pk_max_u16(mag, xv[q][s][e] & 0x7FFF7FFFu);
    }
    mag = max(mag & 0xFFFFu, mag >> 16) << 16;
    const int p = scale_exponent(column_max(mag));
    back = pow2(p);
    const float down = pow2(-p);
#pragma unroll
    for (int q = 0; q < NC; ++q)
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = xv[q][s][e];
          f[2 * e] = bf16_lo(w);
          f[2 * e + 1] = bf16_hi(w);
        }
        xb[q][s] = pack_f16(f, down);
      }
  };
  load_tokens(wave * NC);
  const int active = route_all<NI>(a, sh_ids, sh_w, sh_flag, sh_list, &sh_active);
  const int tiles = a.I >> 4, units = active * tiles;
  const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
  if (u0 >= u1) return;
  const int s0 = 2 * u0, s1 = 2 * u1;                     // steps: tile 2 u is gate, 2 u + 1 is up
  // where the stream stands: a step, its unit's expert and tile, the tile's first
  // row; kept by counting (divisions and LDS reads only where the expert changes)
  struct Pos {
    int s, slot, tile;
    int64_t row;
  };
  auto set_row = [&](Pos& p) {
    const int e = __builtin_amdgcn_readfirstlane(sh_list[p.slot]);
    p.row = (int64_t)e * 2 * a.I + (p.s & 1 ? a.I : 0) + 16 * p.tile;
  };
  auto pos_of = [&](int s) {
    Pos p;
    p.s = s;
    p.slot = (s >> 1) / tiles;
    p.tile = (s >> 1) - p.slot * tiles;
    set_row(p);
    return p;
  };
  auto advance = [&](Pos& p) {                            // stays at the last step
    if (p.s + 1 >= s1) return;
    ++p.s;
    if (p.s & 1) {
      p.row += a.I;
    } else if (++p.tile < tiles) {
      p.row += 16 - (int64_t)a.I;
    } else {
      p.tile = 0;
      ++p.slot;
      set_row(p);
    }
  };

  for (int ph = 0; ph < phases; ++ph) {
    const int c0 = (ph * W + wave) * NC, words = 4 * W * NC;
    int srow[NC], sword[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int it = tid + i * blockDim.x;
      srow[i] = it / words;
      sword[i] = it - srow[i] * words;
    }
    uint32_t sv[D + 1][NC];                               // the last entry: the first step's
    auto load_scales = [&](const Pos& p, int slot) {
      const uint8_t* const base = a.w13_scales + p.row * nb;
#pragma unroll
      for (int i = 0; i < NC; ++i)
        sv[slot][i] = load_scale_word(base + (int64_t)srow[i] * nb, 4 * ph * W * NC + sword[i], nb);
    };
    auto store_scales = [&](int s, int slot) {
#pragma unroll
      for (int i = 0; i < NC; ++i) scl[((s & 1) * 16 + srow[i]) * spitch + sword[i]] = sv[slot][i];
    };
    auto copy_tile = [&](const Pos& p, int slot) {
      const uint8_t* const base = a.w13_packed + p.row * pitch;
#pragma unroll
      for (int q = 0; q < NC; ++q) st4_copy(base, pitch, 15, c0 + q, ring + (slot * NC + q) * kSt4Bytes, lane);
    };
    // the scales travel one tile ahead of the copies (see int4_gemm.hip)
    Pos next = pos_of(s0);                                // the step whose scales are fetched next
    load_scales(next, D);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const Pos here = next;
      advance(next);
      load_scales(next, d);
      copy_tile(here, d);
    }
    store_scales(s0, D);
    if (PASSES && ph > 0)
      load_tokens(c0);
    else
      for (int s = tid; s < active; s += blockDim.x) sh_gs[s] = a.w13_gs[sh_list[s]];
    st4_barrier();

    f32x4 gate;
    auto step = [&](int s, int slot) {
      __builtin_amdgcn_s_waitcnt(st4_vm((D - 1) * 3 * NC));
      __asm__ volatile("" ::: "memory");
      u32x4 w[NC][2];
      uint32_t sw[NC];
#pragma unroll
      for (int q = 0; q < NC; ++q) {
        w[q][0] = st4_read(ring + (slot * NC + q) * kSt4Bytes, r, 2 * g);
        w[q][1] = st4_read(ring + (slot * NC + q) * kSt4Bytes, r, 2 * g + 1);
        sw[q] = scl[((s & 1) * 16 + r) * spitch + 4 * (wave * NC + q) + g];
      }
      __builtin_amdgcn_s_waitcnt(kSt4Lgkm0);
      __asm__ volatile("" ::: "memory");
      store_scales(s + 1, slot);
      const Pos here = next;
      advance(next);
      load_scales(next, slot);
      copy_tile(here, slot);
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < NC; ++q) acc = chunk_product<false>(w[q][0], w[q][1], sw[q], xb[q], nullptr, acc);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] *= back;
      // the gate's sums wait in registers: between two units' writes to red lies
      // the barrier of the second one's gate step
      if (s & 1) {
        *reinterpret_cast<f32x4*>(red + wave * 512 + 4 * lane) = gate;
        *reinterpret_cast<f32x4*>(red + wave * 512 + 256 + 4 * lane) = acc;
      } else {
        gate = acc;
      }
      st4_barrier();
    };
    // the unit's sums: element 4 l + v is lane l's v: token l % 16, column 4 (l / 16) + v of the tile
    int fslot = s0 / 2 / tiles, ftile = s0 / 2 - fslot * tiles, pair = -2;
    auto finish = [&](int u) {
      // this thread's token keeps its pair while the expert stays (threads i and i + 64 k have one token)
      if (pair == -2) {
        pair = -1;
        const int t = (tid >> 2) & 15, e = sh_list[fslot];
        if (t < a.T)
          for (int j = 0; j < a.topk; ++j)
            if (sh_ids[t * a.topk + j] == e) pair = t * a.topk + j;
      }
      for (int i = tid; i < 256; i += blockDim.x) {
        const int n = 4 * (i >> 6) + (i & 3);
        float sum[2] = {0.0f, 0.0f};
        for (int v = 0; v < W; v += 4) {
          float q[4][2];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            q[b][0] = red[min(v + b, W - 1) * 512 + i];
            q[b][1] = red[min(v + b, W - 1) * 512 + 256 + i];
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            sum[0] += v + b < W ? q[b][0] : 0.0f;
            sum[1] += v + b < W ? q[b][1] : 0.0f;
          }
        }
        if (PASSES) {
          float* const h = held + (u - u0) * 512 + i;
          if (ph > 0) {
            sum[0] += h[0];
            sum[1] += h[256];
          }
          if (ph + 1 < phases) {
            h[0] = sum[0];
            h[256] = sum[1];
            continue;
          }
        }
        if (pair < 0) continue;
        const float gs = sh_gs[fslot];
        const float gv = sum[0] * gs, uv = sum[1] * gs;
        a.act[(int64_t)pair * act_pitch(a.I) + 16 * ftile + n] = gv / (1.0f + expf(-gv)) * uv;
      }
      if (++ftile == tiles) {
        ftile = 0;
        ++fslot;
        pair = -2;
      }
    };
    static_assert(D == 2, "two steps a unit and two tiles in flight");
    for (int s = s0; s < s1; s += 2) {
      step(s, 0);
      step(s + 1, 1);
      finish(s >> 1);
    }
    __builtin_amdgcn_s_waitcnt(st4_vm(0));
    __syncthreads();
  }
}

// Down: units (expert, slice of I of W chunks, 16 output columns) in contiguous
// runs; each leaves w[t, j] W2_e a over its slice in parts[slice][pair][column].
// A workgroup counts its units' columns when it is done; whoever completes a
// column tile's count adds its parts, in order of slice and slot.
template <int NC>
__global__ __launch_bounds__(1024) void moe_stream_down_kernel(MoeDecodeArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds8[];
  __shared__ int32_t sh_ids[kMdMaxPairs];
  __shared__ float sh_w[kMdMaxPairs];
  __shared__ int32_t sh_list[kMdMaxPairs];
  __shared__ int32_t sh_done[1024];
  constexpr int D = kMdDepth;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int W = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int K = a.I, nb = K >> 4, nch = (K + kSt4Chunk - 1) / kSt4Chunk, P = a.T * a.topk;
  const int64_t pitch = K >> 1;
  uint8_t* const ring = lds8 + wave * (D * NC * kSt4Bytes);
  float* const red = reinterpret_cast<float*>(lds8 + W * (D * NC * kSt4Bytes));          // [2][W][256]
  const int spitch = md_scale_pitch(W * NC);
  uint32_t* const scl = reinterpret_cast<uint32_t*>(red + 2 * W * 256);                  // [2][16][spitch]

  const int active = *a.active, slices = a.slices, tiles = a.H >> 4;
  for (int p = tid; p < P; p += blockDim.x) {             // of the list, the first `active` hold experts
    sh_ids[p] = a.ids[p];
    sh_w[p] = a.weights[p];
    sh_list[p] = a.list[p];
  }
  __syncthreads();
  const int units = active * slices * tiles;
  const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
  if (active == 0) {                                       // no token has an expert
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + tid; i < (int64_t)a.T * a.H; i += (int64_t)gridDim.x * blockDim.x)
      a.out[i] = 0;
    return;
  }
  if (u0 >= u1) return;
  // where the stream stands (see the up kernel); combo = (expert slot, slice)
  struct Pos {
    int u, combo, slice, tile;
    int64_t row;
  };
  auto set_row = [&](Pos& p) {
    const int slot = p.combo / slices;
    p.slice = p.combo - slot * slices;
    p.row = (int64_t)__builtin_amdgcn_readfirstlane(sh_list[slot]) * a.H + 16 * p.tile;
  };
  auto pos_of = [&](int u) {
    Pos p;
    p.u = u;
    p.combo = u / tiles;
    p.tile = u - p.combo * tiles;
    set_row(p);
    return p;
  };
  auto advance = [&](Pos& p) {
    if (p.u + 1 >= u1) return;
    ++p.u;
    if (++p.tile < tiles) {
      p.row += 16;
    } else {
      p.tile = 0;
      ++p.combo;
      set_row(p);
    }
  };
  const int words = 4 * W * NC;
  int srow[NC], sword[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int it = tid + i * blockDim.x;
    srow[i] = it / words;
    sword[i] = it - srow[i] * words;
  }
  uint32_t sv[D + 1][NC];                                 // the last entry: the first unit's
  int sslice[D + 1];
  // 32-bit offsets from the tile's first row: 16 rows of I / 2 bytes, I <= 2^29
  auto load_scales = [&](const Pos& p, int slot) {
    const uint8_t* const base = a.w2_scales + p.row * nb;
    sslice[slot] = p.slice;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      sv[slot][i] = reinterpret_cast<const Word4A1*>(
                        base + (uint32_t)(srow[i] * nb + scale_word_offset(words * p.slice + sword[i], nb)))->v;
  };
  // the word is cut when it is stored, a step later: here it would have to be waited for
  auto store_scales = [&](int u, int slot) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      scl[((u & 1) * 16 + srow[i]) * spitch + sword[i]] = scale_word(sv[slot][i], words * sslice[slot] + sword[i], nb);
  };
  const uint32_t roff = (uint32_t)(lane >> 3) * (uint32_t)pitch;
  auto copy_tile = [&](const Pos& p, int slot) {
    const uint8_t* const base = a.w2_packed + p.row * pitch;
#pragma unroll
    for (int q = 0; q < NC; ++q) {
      const uint32_t off = roff + (uint32_t)st4_offset<int>((p.slice * W + wave) * NC + q, (int)pitch, lane);
      st4_copy_rows(base + off, base + 8 * pitch + off, ring + (slot * NC + q) * kSt4Bytes);
    }
  };
  Pos next = pos_of(u0), now = next;                       // fetched next; computed now
  load_scales(next, D);
#pragma unroll
  for (int d = 0; d < D; ++d) {
    const Pos here = next;
    advance(next);
    load_scales(next, d);
    copy_tile(here, d);
  }
  store_scales(u0, D);
  st4_barrier();

  f16x8 xb[NC][8], xr[NC][8];
  float back = 0.0f;
  int out_pair = -1;                                       // of this thread's token in the sums
  // the activations of (expert, slice) c: column r is token r's pair with the expert, or zeros
  auto load_act = [&](const Pos& at) {
    const int e = sh_list[at.combo / slices], c0 = (at.slice * W + wave) * NC;
    int pair = -1;
    out_pair = -1;
    if (r < a.T)
      for (int j = 0; j < a.topk; ++j)
        if (sh_ids[r * a.topk + j] == e) pair = r * a.topk + j;
    const int ot = (tid >> 2) & 15;
    if (ot < a.T)
      for (int j = 0; j < a.topk; ++j)
        if (sh_ids[ot * a.topk + j] == e) out_pair = ot * a.topk + j;
    const float* const act = a.act + (int64_t)max(pair, 0) * act_pitch(K) + 64 * g;
    uint32_t mag = 0;
    float f[NC][8][8];
#pragma unroll
    for (int q = 0; q < NC; ++q) {
      // rows are padded to whole chunks: what lies past K, or belongs to no pair, is replaced by zeros
      const float* const row = act + (int64_t)kSt4Chunk * min(c0 + q, nch - 1);
      const int have = pair >= 0 ? K - kSt4Chunk * (c0 + q) - 64 * g : 0;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const f32x4 lo = *reinterpret_cast<const f32x4*>(row + 8 * s), hi = *reinterpret_cast<const f32x4*>(row + 8 * s + 4);
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2) {
          f[q][s][e2] = 8 * s < have ? lo[e2] : 0.0f;
          f[q][s][4 + e2] = 8 * s < have ? hi[e2] : 0.0f;
          mag = max(mag, max(__float_as_uint(f[q][s][e2]) & 0x7FFFFFFFu, __float_as_uint(f[q][s][4 + e2]) & 0x7FFFFFFFu));
        }
      }
    }
    const int p = scale_exponent(column_max(mag));
    back = pow2(p) * a.w2_gs[e] * (pair >= 0 ? sh_w[pair] : 0.0f);
    const float down = pow2(-p);
#pragma unroll
    for (int q = 0; q < NC; ++q)
#pragma unroll
      for (int s = 0; s < 8; ++s) xb[q][s] = pack_f16_pair(f[q][s], down, &xr[q][s]);
  };

  auto step = [&](int u, int slot) {
    __builtin_amdgcn_s_waitcnt(st4_vm((D - 1) * 3 * NC));
    __asm__ volatile("" ::: "memory");
    u32x4 w[NC][2];
    uint32_t sw[NC];
#pragma unroll
    for (int q = 0; q < NC; ++q) {
      w[q][0] = st4_read(ring + (slot * NC + q) * kSt4Bytes, r, 2 * g);
      w[q][1] = st4_read(ring + (slot * NC + q) * kSt4Bytes, r, 2 * g + 1);
      sw[q] = scl[((u & 1) * 16 + r) * spitch + 4 * (wave * NC + q) + g];
    }
    __builtin_amdgcn_s_waitcnt(kSt4Lgkm0);
    __asm__ volatile("" ::: "memory");
    store_scales(u + 1, slot);
    const Pos here = next;
    advance(next);
    load_scales(next, slot);
    copy_tile(here, slot);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < NC; ++q) acc = chunk_product<true>(w[q][0], w[q][1], sw[q], xb[q], xr[q], acc);
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] *= back;
    *reinterpret_cast<f32x4*>(red + ((u & 1) * W + wave) * 256 + 4 * lane) = acc;
    st4_barrier();
    for (int i = tid; i < 256; i += blockDim.x) {
      if (out_pair < 0) break;                             // threads i and i + 64 k have one token
      const int n = 4 * (i >> 6) + (i & 3);
      const float* const part = red + (u & 1) * W * 256 + i;
      float sum = 0.0f;
      for (int v = 0; v < W; v += 4) {
        float q[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) q[b] = part[min(v + b, W - 1) * 256];
#pragma unroll
        for (int b = 0; b < 4; ++b) sum += v + b < W ? q[b] : 0.0f;
      }
      __hip_atomic_store(a.parts + ((int64_t)now.slice * P + out_pair) * a.H + 16 * now.tile + n, sum,
                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    advance(now);
  };
  // runs of one (expert, slice); a unit's ring slot is its parity in the workgroup's run
  for (int u = u0; u < u1;) {
    const int end = min(u1, u + tiles - now.tile);
    load_act(now);
    if ((u - u0) & 1) step(u++, 1);
    for (; u + 1 < end; u += 2) {
      step(u, 0);
      step(u + 1, 1);
    }
    if (u < end) step(u++, 0);
  }

  // count the units; a tile is complete with active * slices of them.  The parts
  // were stored past the caches (agent scope) and have arrived once this wait
  // ends, so the counting needs no cache write-back, only order
  __builtin_amdgcn_s_waitcnt(st4_vm(0));
  __syncthreads();
  for (int v0 = u0; v0 < u1; v0 += 1024) {
    const int n = min(1024, u1 - v0);
    for (int i = tid; i < n; i += blockDim.x) {
      const int tile = (v0 + i) % tiles;
      const int before = __hip_atomic_fetch_add(a.counters + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      sh_done[i] = before + 1 == active * slices ? tile : -1;
    }
    __syncthreads();
    // the complete tiles' outputs, two columns a thread, read past the caches as
    // they were written (a fence that empties the caches instead: 20 us more)
    const int halves = 8 * a.T, terms = a.topk * slices;
    for (int o = tid; o < n * halves; o += blockDim.x) {
      const int i = o / halves, q = o - i * halves, t = q >> 3, tile = sh_done[i];
      if (tile < 0) continue;
      const int n0 = 16 * tile + 2 * (q & 7);
      float sum[2] = {0.0f, 0.0f};
      for (int c = 0; c < terms; c += 8) {                // eight loads at a time, added in order
        uint64_t v[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const int k = min(c + b, terms - 1), j = k / slices, p = t * a.topk + j;
          v[b] = __hip_atomic_load(
              reinterpret_cast<const uint64_t*>(a.parts + ((int64_t)(k - j * slices) * P + p) * a.H + n0),
              __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const int k = min(c + b, terms - 1);
          if (c + b < terms && sh_ids[t * a.topk + k / slices] >= 0) {
            sum[0] += __uint_as_float((uint32_t)v[b]);
            sum[1] += __uint_as_float((uint32_t)(v[b] >> 32));
          }
        }
      }
      *reinterpret_cast<uint32_t*>(a.out + (int64_t)t * a.H + n0) =
          __builtin_bit_cast(uint32_t, bf16x2{(__bf16)sum[0], (__bf16)sum[1]});
    }
    __syncthreads();
  }
}

namespace {

int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }

// Workgroups that share one output tile's K: enough for one per compute unit.
int64_t down_split(int64_t H) {
  const int64_t tiles = H / 16;
  return std::max<int64_t>(1, std::min<int64_t>(8, 256 / tiles));
}

}  // namespace

namespace {

// Streamed form: chunks per wavefront and wavefronts over K, and passes over it.
struct StreamPlan {
  int nc, waves, passes;
};
StreamPlan stream_plan(int64_t K) {
  const int64_t nch = (K + kSt4Chunk - 1) / kSt4Chunk;
  const int64_t passes = (nch + 15) / 16;
  return StreamPlan{1, (int)((nch + passes - 1) / passes), (int)passes};
}

bool streamed(int64_t H, int64_t I) { return H % 32 == 0 && I % 32 == 0 && H >= 64 && I >= 64; }

}  // namespace

int64_t moe_decode_workspace_bytes(int64_t T, int64_t topk, int64_t H, int64_t I) {
  const int64_t P = T * topk, split = down_split(H);
  const int64_t parts = streamed(H, I) ? stream_plan(I).passes * P * H * 4
                                       : (split > 1 ? H / 16 * split * 256 * 4 : 0);
  return 3 * up256(P * 4) + 256 + up256(P * act_pitch(I) * 4) + up256(H / 16 * 4) + parts;
}

namespace {

template <int NI>
hipError_t launch_stream_up(const MoeDecodeArgs& a, int64_t active, hipStream_t stream) {
  const StreamPlan p = stream_plan(a.H);
  const int dev = current_device();
  const void* const fn = p.passes > 1 ? (const void*)moe_stream_up_kernel<NI, 1, true>
                                      : (const void*)moe_stream_up_kernel<NI, 1, false>;
  int64_t lds = (int64_t)p.waves * (kMdDepth * kSt4Bytes + 2048) + 128 * md_scale_pitch(p.waves);
  const int64_t units = active * (a.I / 16);
  int64_t grid;
  if (p.passes > 1) {                                     // one workgroup a compute unit; its units' held sums fit beside
    const int64_t room = std::max<int64_t>(1, (144 * 1024 - lds) / 2048);
    grid = std::max<int64_t>(std::min<int64_t>(units, device_cus(dev)), (units + room - 1) / room);
    lds += (units + grid - 1) / grid * 2048;
  }
  const hipError_t e = ensure_dynamic_lds(fn, dev, (int)lds);
  if (e != hipSuccess) return e;
  if (p.passes == 1)
    grid = std::min<int64_t>(units, (int64_t)device_cus(dev) * blocks_per_cu(fn, dev, 64 * p.waves, (size_t)lds));
  return launch_kernel_lds(fn, dim3((unsigned)grid), dim3(64 * p.waves), (size_t)lds, stream, a);
}

hipError_t launch_stream(MoeDecodeArgs a, int64_t active, hipStream_t stream) {
  const StreamPlan p = stream_plan(a.I);
  a.slices = p.passes;
  a.n_counters = a.H / 16;
  hipError_t e = a.E <= 64    ? launch_stream_up<1>(a, active, stream)
                 : a.E <= 256 ? launch_stream_up<4>(a, active, stream)
                              : launch_stream_up<16>(a, active, stream);
  if (e != hipSuccess) return e;
  const int dev = current_device();
  const void* const fn = (const void*)moe_stream_down_kernel<1>;
  const int64_t lds = (int64_t)p.waves * (kMdDepth * kSt4Bytes + 2048) + 128 * md_scale_pitch(p.waves);
  e = ensure_dynamic_lds(fn, dev, (int)lds);
  if (e != hipSuccess) return e;
  const int64_t units = active * p.passes * (a.H / 16);
  const int64_t grid =
      std::min<int64_t>(units, (int64_t)device_cus(dev) * blocks_per_cu(fn, dev, 64 * p.waves, (size_t)lds));
  return launch_kernel_lds(fn, dim3((unsigned)grid), dim3(64 * p.waves), (size_t)lds, stream, a);
}

}  // namespace

hipError_t launch_moe_decode(MoeDecodeArgs a, void* workspace, hipStream_t stream) {
  const int64_t P = (int64_t)a.T * a.topk;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  auto take = [&](int64_t bytes) {
    uint8_t* const at = p;
    p += up256(bytes);
    return at;
  };
  a.ids = reinterpret_cast<int32_t*>(take(P * 4));
  a.weights = reinterpret_cast<float*>(take(P * 4));
  a.list = reinterpret_cast<int32_t*>(take(P * 4));
  a.active = reinterpret_cast<int32_t*>(take(4));
  a.act = reinterpret_cast<float*>(take(P * act_pitch(a.I) * 4));
  a.a_hi = reinterpret_cast<uint16_t*>(a.act);
  a.a_lo = a.a_hi + P * a.I;
  a.counters = reinterpret_cast<int32_t*>(take(a.H / 16 * 4));
  a.parts = reinterpret_cast<float*>(p);
  const int64_t active = std::min<int64_t>(a.E, P), tiles = a.I / 16;   // chosen experts at most
  if (streamed(a.H, a.I)) return launch_stream(a, active, stream);
  a.down_split = (int)down_split(a.H);
  a.n_counters = a.down_split > 1 ? a.H / 16 : 0;
  // K split over 1, 2 or 4 wavefronts until the wavefronts fill the GPU
  // (sixteen for each of 256 compute units)
  const int64_t nch = (a.H + kMdChunk - 1) / kMdChunk;
  int splitk = 1;
  while (splitk < kMdWaves && active * tiles * splitk < 4096 && 2 * splitk <= nch) splitk *= 2;
  a.splitk = splitk;
  const int64_t per = kMdWaves / splitk, items = active * ((tiles + per - 1) / per);
  const void* fn = a.E <= 64    ? (const void*)moe_decode_up_kernel<1>
                   : a.E <= 256 ? (const void*)moe_decode_up_kernel<4>
                                : (const void*)moe_decode_up_kernel<16>;
  hipError_t e = launch_kernel(fn, dim3((unsigned)std::min<int64_t>(items, 1024)), dim3(64 * kMdWaves), stream, a);
  if (e != hipSuccess) return e;
  return launch_kernel((const void*)moe_decode_down_kernel, dim3((unsigned)(a.H / 16 * a.down_split)),
                       dim3(64 * kMdDownWaves), stream, a);
}

}  // namespace nvfp4
