// The whole W4A16 NVFP4 expert layer for a few tokens (T <= 16), from the
// router's logits, in two kernels (gfx950).
//
// Weights as in nvfp4_moe.hip (vLLM modelopt.py, ModelOptNvFp4FusedMoE,
// use_a16).  For token t the router's scores are softmax or sigmoid of its
// logits, the topk largest logits (of score + bias, with a bias) are chosen,
// equal ones by the lower index, and
//   out[t] = sum_j w[t, j] W2_e (silu(W1_e x[t]) * (W3_e x[t])),  e = ids[t, j].
//
// moe_decode_up_kernel: every workgroup routes all tokens by itself (a few
//   hundred logits, one wavefront per token; cheaper than a launch), lists the
//   chosen experts in order and walks its share of (expert, 16 columns of I):
//   one wavefront holds the gate and the up rows of the same 16 columns, so
//   the activation is applied in its registers.
// moe_decode_down_kernel: a workgroup owns 16 output columns; its wavefronts
//   split the K = I of all chosen experts, each expert's sum is weighted by
//   w[t, j] as it ends, so nothing per pair is written.
//
// The MFMA's columns are the tokens themselves (16 at most), a token that did
// not choose the expert is a column of zeros: no gathering, no lists of pairs.
// Weights stream straight to registers, one 256-k chunk ahead: lane (r, g) =
// (lane % 16, lane / 16) holds row r's codes of k = 256 c + 64 g + [0, 64) (two
// 16-byte loads) and their four block scales (one 4-byte load); MFMA step s
// multiplies k = 64 g + 8 s + [0, 8) of each g.  A code times its block scale is
// exact in bf16.  The hidden activation is kept as a bf16 pair hi + lo (16 bits
// of it), so that the only rounding to bf16 is the output's.
#include <algorithm>

#include "nvfp4_device.hpp"
#include "nvfp4_launch.hpp"

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
  const int pairs = a.T * a.topk;
  for (int e = tid; e < 64 * NI; e += 64 * kMdWaves) sh_flag[e] = 0;
  for (int t = wave; t < a.T; t += kMdWaves) route_token<NI>(a, t, lane, sh_ids, sh_w);
  __syncthreads();
  for (int p = tid; p < pairs; p += 64 * kMdWaves)
    if (sh_ids[p] >= 0) sh_flag[sh_ids[p]] = 1;
  __syncthreads();
  if (wave == 0) {                                      // the chosen experts in increasing order
    int n = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool on = sh_flag[64 * i + lane] != 0;
      const uint64_t all = __ballot(on);
      if (on) sh_list[n + __popcll(all & (((uint64_t)1 << lane) - 1))] = 64 * i + lane;
      n += __popcll(all);
    }
    if (lane == 0) sh_active = n;
  }
  __syncthreads();
  const int active = sh_active;
  if (blockIdx.x == 0) {                                // for the second kernel and the caller
    for (int p = tid; p < pairs; p += 64 * kMdWaves) {
      a.ids[p] = sh_ids[p];
      a.weights[p] = sh_w[p];
      if (a.ids_out) a.ids_out[p] = sh_ids[p];
      if (a.weights_out) a.weights_out[p] = sh_w[p];
    }
    for (int s = tid; s < active; s += 64 * kMdWaves) a.list[s] = sh_list[s];
    if (tid == 0) *a.active = active;
    for (int i = tid; i < a.n_counters; i += 64 * kMdWaves) a.counters[i] = 0;
  }

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

namespace {

int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }

// Workgroups that share one output tile's K: enough for one per compute unit.
int64_t down_split(int64_t H) {
  const int64_t tiles = H / 16;
  return std::max<int64_t>(1, std::min<int64_t>(8, 256 / tiles));
}

}  // namespace

int64_t moe_decode_workspace_bytes(int64_t T, int64_t topk, int64_t H, int64_t I) {
  const int64_t P = T * topk, split = down_split(H);
  return 3 * up256(P * 4) + 256 + 2 * up256(P * I * 2) + up256(H / 16 * 4) +
         (split > 1 ? H / 16 * split * 256 * 4 : 0);
}

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
  a.a_hi = reinterpret_cast<uint16_t*>(take(P * a.I * 2));
  a.a_lo = reinterpret_cast<uint16_t*>(take(P * a.I * 2));
  a.counters = reinterpret_cast<int32_t*>(take(a.H / 16 * 4));
  a.parts = reinterpret_cast<float*>(p);
  a.down_split = (int)down_split(a.H);
  a.n_counters = a.down_split > 1 ? a.H / 16 : 0;
  // chosen experts at most; K split over 1, 2 or 4 wavefronts until the
  // wavefronts fill the GPU (sixteen for each of 256 compute units)
  const int64_t active = std::min<int64_t>(a.E, P), tiles = a.I / 16;
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
