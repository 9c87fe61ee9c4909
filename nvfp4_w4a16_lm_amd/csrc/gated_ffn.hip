// Gated feed-forward block on bf16 weights (gfx950), forward and backward.
//
//   [g, u] = x W13^T,  a = silu(g) u,  y = a W2^T
//   da = dy W2,  du = da silu(g),  dg = da u silu'(g),  silu'(g) = s + g s (1 - s), s = 1 / (1 + e^-g)
//   dx = [dg, du] W13,  dW13 = [dg, du]^T x,  dW2 = dy^T a
//
// Forward: both projections, the activation and the product are one kernel
// whose tile holds matching rows of the gate and the up projection; the
// activation enters the down projection rounded to bf16, up to 16 tokens as a pair
// of bf16.  Kept for the
// backward pass: h = [g, u] in float32 and a in bf16, as the operand of dW2 that it
// is.  (With h in bf16 the gradients of x and W13 are off by 0.0030 of their norm instead
// of 0.0024, where one rounding of the result is 0.0017; the step of 4096 tokens is 4 % faster.)  Backward:
// the kernel of da = dy W2 ends in [dg, du], in bf16 as operands; then three products.
//
// Measured: one token of (4096, 14336) 69 us (5.1 TB/s: 43 us both projections at 5.5 TB/s, 22 the down projection in
// 16 parts, 5 their join), 16 tokens 72 us; the step of 4096 tokens 3.4 ms (1.26 PFLOP/s: 0.85, 0.37, 0.54, 0.43,
// 0.73, 0.77 ms in the order above); of 333 tokens of (2080, 5616) 153 us on inputs in the last-level cache, 175 us from
// memory.  Small I: both projections are a workgroup for 64 columns, one token of (4096, 1408) 40 us, floor 7.
#include "dense_tile.hpp"

namespace nvfp4 {

// Sum of `splits` partial products: out bf16 [M][N] from float [splits][M][N].
__global__ __launch_bounds__(256) void gated_join_kernel(const float* __restrict__ parts, int64_t count, int splits,
                                                         uint16_t* __restrict__ out) {
  const int64_t i = 8 * ((int64_t)blockIdx.x * 64 + (threadIdx.x & 63));
  float v[8];
  tile_join(parts, i, count, splits, i < count, v);
  if (threadIdx.x < 64 && i < count) *reinterpret_cast<u32x4*>(out + i) = pack8(v);
}

// The down projection and dx: K split where the tiles are few, at least 8 steps a part.
static TileSplit gated_split(int64_t M, int64_t N, int64_t K) { return tile_split(M, N, K, 8, 16); }
static int64_t gated_split_floats(int64_t M, int64_t N, int64_t K) { return tile_split_floats(M, N, K, 8, 16); }

struct GatedLayout {
  int64_t parts, bytes;
};
// Up to 16 tokens the activation enters the down projection as a pair of bf16, 16 bits of it: its second rows fill
// the tile of 32 (one token 67.2 us rounded to bf16, 67.6 so; 16 tokens 70.6, 71.2).
constexpr int64_t kGatedPair = 16;

// No part's size falls as T grows, though the pair ends and the splits change: a workspace kept for the largest batch
// holds every smaller one.
static GatedLayout gated_layout(int64_t T, int64_t H, int64_t I, bool backward) {
  GatedLayout l = {};
  const int64_t pairs = T < kGatedPair ? T : kGatedPair;
  // the forward pass's a, for few tokens a pair, and the backward's [dg, du] share a place
  const int64_t rows = backward ? 2 * T : T > 2 * pairs ? T : 2 * pairs;
  l.parts = up256(2 * rows * I);
  // the joined products: of a pair always, else where K is split
  const int64_t split = gated_split_floats(T, H, backward ? 2 * I : I);
  l.bytes = l.parts + up256(4 * (split > pairs * H ? split : pairs * H));
  return l;
}

int64_t gated_ffn_workspace_bytes(int64_t T, int64_t H, int64_t I, bool backward) {
  const int64_t b = T == 0 ? 16 : gated_layout(T, H, I, backward).bytes;
  return b < 16 ? 16 : b;
}

// out bf16 [M, N] = q [M, K] p^T or q p (PT), K split where the tiles are few; with `pair` q has M rows more, whose
// products are added
template <bool PT>
static hipError_t gated_product(const void* q, const void* p, int64_t M, int64_t N, int64_t K, bool pair, void* out,
                                float* parts, hipStream_t stream) {
  const int64_t rows = pair ? 2 * M : M;
  TileArgs a = {};
  a.p = (const uint8_t*)p;
  a.q = (const uint8_t*)q;
  a.p_pitch = 2 * (PT ? N : K);
  a.q_pitch = 2 * K;
  a.p_rows = PT ? K : N;
  a.q_rows = rows;
  a.M = (int)rows;
  a.N = (int)N;
  a.K = (int)K;
  a.out_pitch = N;
  a.pair_rows = pair ? (int)M : 0;
  const TileSplit s = gated_split(rows, N, K);
  a.k_split = s.k_split;
  a.splits = s.splits;
  if (a.splits == 1 && !pair) {
    a.out = out;
    return launch_tile<kTileBf16, PT, false>(a, s.size, stream);
  }
  a.out = parts;
  const hipError_t e = launch_tile<kTileF32, PT, false>(a, s.size, stream);
  if (e != hipSuccess) return e;
  return launch_kernel((const void*)gated_join_kernel, dim3((unsigned)((M * N / 8 + 63) / 64)), dim3(256), stream,
                       (const float*)parts, (int64_t)(M * N), (int)a.splits, (uint16_t*)out);
}

// out bf16 [M, N] = q^T p, q [K, M], p [K, N]
static hipError_t gated_weight_grad(const void* q, int64_t M, const void* p, int64_t N, int64_t K, void* out,
                                    hipStream_t stream) {
  TileArgs a = {};
  a.p = (const uint8_t*)p;
  a.q = (const uint8_t*)q;
  a.p_pitch = 2 * N;
  a.q_pitch = 2 * M;
  a.p_rows = a.q_rows = K;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.splits = 1;
  a.k_split = (int)((K + 63) / 64 * 64);
  a.out = out;
  a.out_pitch = N;
  return launch_tile<kTileBf16, true, true>(a, tile_size(M, N, (K + 63) / 64, 1, true), stream);
}

hipError_t launch_gated_ffn(const void* x, int64_t T, int64_t H, const void* w13, const void* w2, int64_t I,
                            float* h, void* act, void* workspace, void* y, hipStream_t stream) {
  const GatedLayout l = gated_layout(T, H, I, false);
  uint8_t* const ws = (uint8_t*)workspace;
  TileArgs a = {};
  a.p = (const uint8_t*)w13;
  a.q = (const uint8_t*)x;
  a.p_pitch = a.q_pitch = 2 * H;
  a.p_rows = 2 * I;
  a.q_rows = T;
  a.M = (int)T;
  a.N = (int)I;
  a.I = (int)I;
  a.K = (int)H;
  a.splits = 1;
  a.k_split = (int)((H + 63) / 64 * 64);
  const bool pair = T <= kGatedPair;
  a.out = act == nullptr || pair ? ws : act;
  a.out_pitch = I;
  a.pair_rows = pair ? (int)T : 0;
  a.act = pair ? (uint16_t*)act : nullptr;
  a.h = h;
  const hipError_t e = launch_tile<kTileGated, false, false>(a, tile_size(T, 2 * I, (H + 63) / 64, 1), stream);
  if (e != hipSuccess) return e;
  return gated_product<false>(a.out, w2, T, H, I, pair, y, (float*)(ws + l.parts), stream);
}

hipError_t launch_gated_ffn_backward(const void* x, int64_t T, int64_t H, const float* h, const void* act,
                                     const void* w13, const void* w2, int64_t I, const void* dy, void* workspace,
                                     void* dx, void* dw13, void* dw2, hipStream_t stream) {
  const GatedLayout l = gated_layout(T, H, I, true);
  uint8_t* const ws = (uint8_t*)workspace;
  TileArgs a = {};
  a.p = (const uint8_t*)w2;
  a.q = (const uint8_t*)dy;
  a.p_pitch = 2 * I;
  a.q_pitch = 2 * H;
  a.p_rows = H;
  a.q_rows = T;
  a.M = (int)T;
  a.N = (int)I;
  a.I = (int)I;
  a.K = (int)H;
  a.splits = 1;
  a.k_split = (int)((H + 63) / 64 * 64);
  a.h = const_cast<float*>(h);
  a.dh = (uint16_t*)ws;
  hipError_t e = launch_tile<kTileGatedBack, true, false>(a, tile_size(T, I, (H + 63) / 64, 1), stream);
  if (e != hipSuccess) return e;
  if (dw2 != nullptr) {
    e = gated_weight_grad(dy, H, act, I, T, dw2, stream);
    if (e != hipSuccess) return e;
  }
  if (dx != nullptr) {
    e = gated_product<true>(ws, w13, T, H, 2 * I, false, dx, (float*)(ws + l.parts), stream);
    if (e != hipSuccess) return e;
  }
  return dw13 == nullptr ? hipSuccess : gated_weight_grad(ws, 2 * I, x, H, T, dw13, stream);
}

}  // namespace nvfp4
