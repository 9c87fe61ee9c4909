// Softmax cross entropy from hidden states and the lm_head weight (gfx950), without
// the logits ever in memory, and its gradients.
//
//   z = x W^T + b,  m = max_j z_j,  s = sum_j exp(z_j - m),  lse = m + log s,  loss = (m - z_t) + log s
//   dz_j = (dloss + dlse) exp(z_j - m) / s - dloss 1[j = t]
//   dx = dz W,  dW = dz^T x,  db = sum over rows of dz
//
// dz enters the products rounded to bf16.  A row's target has by far its largest dz, and what rounding takes from it is
// the same share of all it adds to a row of dx and of dW: it is kept (rest) and added to each result.  Gradients are
// then off by 0.0017 of their norm, which is their own rounding (without: 0.0024, 0.0028 of 17 rows, up to 0.0032 of one).
// It costs 0.4 % of the step of 4096 rows, 4 % of that of 333 (243 -> 253 us, in dW).
//
// Rows whose target is outside the vocabulary have no loss and no gradient: the
// rows that count are gathered first, and only they enter the products.
//
// Forward: tiles of logits end as one maximum and one sum per row and tile,
// which a second kernel joins.  Backward, for each piece of the vocabulary: the
// logits again, ending in dz (bf16, the operand type of what follows); dx gains dz W
// in float32; the piece of dW is dz^T x.  A piece's dz is 128 MB at most up to 65536 rows, 2 KB a row beyond.
//
// Measured: loss of 2048 x 128256 x 4096 1.65 ms (1.31 PFLOP/s), with gradients at 4096 rows, 5 % of them
// without a target, 12.9 ms (1.26 PFLOP/s: logits 3.2, again 3.6, dx 3.2, dW 3.2 ms); both bound by the
// card's power.  333 x 32003 x 2080 253 us on inputs in the last-level cache, 279 us from memory.  17 x 32003 x 512
// 44 us: eight launches, whose kernels take 46 us one after the other.
#include "dense_tile.hpp"

namespace nvfp4 {

struct CeGather {
  const uint16_t* x;
  const int32_t* tok;
  int32_t M, V, K;
  int32_t rows;                      // rows a workgroup gathers: four, more beyond 4096 rows, as each counts all before it
  uint16_t* xc;                      // rows that count, in order
  int32_t* ctok;
  int32_t* index;                    // their rows
  int32_t* count;
  // forward: what the other rows get
  float* loss;
  float* lse;
  float2* stats;
  // backward
  const float2* stats_in;
  const float* dloss;
  const float* dlse;
  float2* cstats;
  float2* coef;
  uint16_t* dx;                      // zero in the other rows
};

// Workgroup b: rows a.rows b and on, a wavefront each, four at a time.  A row's place is the number of earlier rows
// that count.
__global__ __launch_bounds__(256) void ce_gather_kernel(CeGather a) {
  __shared__ int part[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row0 = blockIdx.x * a.rows, row1 = min(row0 + a.rows, a.M);
  int before = 0;
#pragma unroll 8
  for (int i = tid; i < row0; i += 256) before += (uint32_t)a.tok[i] < (uint32_t)a.V;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) before += __shfl_xor(before, d, 64);
  if (lane == 0) part[wave] = before;
  __syncthreads();
  int first = part[0] + part[1] + part[2] + part[3];
  const int pieces = a.K / 8;
  for (int base = row0; base < row1; base += 4) {
    const bool mine = lane < 4 && base + lane < row1 && (uint32_t)a.tok[base + lane] < (uint32_t)a.V;
    const uint32_t rows = (uint32_t)__ballot(mine);
    const int row = base + wave, place = first + __popc(rows & ((1u << wave) - 1));
    first += __popc(rows);
    if (row >= row1) continue;
    if (rows >> wave & 1) {
      const u32x4* const src = reinterpret_cast<const u32x4*>(a.x + (int64_t)row * a.K);
      u32x4* const dst = reinterpret_cast<u32x4*>(a.xc + (int64_t)place * a.K);
#pragma unroll 8
      for (int p = lane; p < pieces; p += 64) dst[p] = src[p];
      if (lane == 0) {
        a.ctok[place] = a.tok[row];
        a.index[place] = row;
        if (a.coef != nullptr) {
          const float d = a.dloss[row];
          a.cstats[place] = a.stats_in[row];
          a.coef[place] = make_float2(d + (a.dlse != nullptr ? a.dlse[row] : 0.0f), d);
        }
      }
    } else {
      if (a.dx != nullptr) {
        u32x4* const dst = reinterpret_cast<u32x4*>(a.dx + (int64_t)row * a.K);
        for (int p = lane; p < pieces; p += 64) dst[p] = u32x4{0, 0, 0, 0};
      }
      if (lane == 0 && a.loss != nullptr) {
        a.loss[row] = 0.0f;
        if (a.lse != nullptr) a.lse[row] = 0.0f;
        a.stats[row] = make_float2(0.0f, 1.0f);
      }
    }
  }
  if (row1 == a.M && tid == 0) *a.count = first;
}

// A wavefront per row joins its tiles' maxima and sums.
__global__ __launch_bounds__(256) void ce_join_kernel(const float2* __restrict__ parts, int tiles,
                                                      const float* __restrict__ tlogit,
                                                      const int32_t* __restrict__ index,
                                                      const int32_t* __restrict__ count, float* __restrict__ loss,
                                                      float* __restrict__ lse, float2* __restrict__ stats) {
  const int lane = threadIdx.x & 63, row = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= *count) return;
  const float2* const p = parts + (int64_t)row * tiles;
  float m = -INFINITY, s = 0.0f;
  for (int i = lane; i < tiles; i += 64) {
    const float2 v = p[i];
    if (v.x > m) {
      if (m != -INFINITY) s *= exp_fast(m - v.x);
      m = v.x;
    }
    s += v.x == -INFINITY ? v.y : v.y * exp_fast(v.x - m);       // -inf: no logit, 0, or NaN
  }
  float mm = m;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mm = fmaxf(mm, __shfl_xor(mm, d, 64));
  if (m != mm && m != -INFINITY) s *= exp_fast(m - mm);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
  if (lane == 0) {
    const int at = index[row];
    const float ls = logf(s);
    loss[at] = tlogit[row] == -INFINITY ? (s == s ? INFINITY : s) : (mm - tlogit[row]) + ls;
    if (lse != nullptr) lse[at] = mm == -INFINITY && s == 0.0f ? -INFINITY : mm + ls;
    stats[at] = make_float2(mm, s);
  }
}

// dx: the splits' sums and the remainder's share of the target's row of W, rounded once, back in their rows; a
// workgroup 512 columns of a row
__global__ __launch_bounds__(256) void ce_dx_kernel(const float* __restrict__ parts, int M, int K, int splits,
                                                    const uint16_t* __restrict__ w, const int32_t* __restrict__ tok,
                                                    const float* __restrict__ rest, const int32_t* __restrict__ index,
                                                    const int32_t* __restrict__ count, uint16_t* __restrict__ dx) {
  const int row = blockIdx.x, k = 8 * (blockIdx.y * 64 + (threadIdx.x & 63));
  if (row >= *count) return;
  const bool mine = threadIdx.x < 64 && k < K;
  u32x4 target = {0, 0, 0, 0};
  if (mine) target = *reinterpret_cast<const u32x4*>(w + (int64_t)tok[row] * K + k);
  float v[8], t[8];
  tile_join(parts, (int64_t)row * K + k, (int64_t)M * K, splits, k < K, v);
  if (!mine) return;
  unpack8(target, t);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += finite_or_0(rest[row] * t[e]);
  *reinterpret_cast<u32x4*>(dx + (int64_t)index[row] * K + k) = pack8(v);
}

// db of a piece: column sums of dz, 64 columns a workgroup, and the targets' remainders.  Hits among 64
// rows' targets are few and added one after the other, in the rows' order.
__global__ __launch_bounds__(256) void ce_bias_kernel(const uint16_t* __restrict__ d, int64_t pitch, int width,
                                                      const int32_t* __restrict__ tok, const float* __restrict__ rest,
                                                      int n_first, const int32_t* __restrict__ count,
                                                      uint16_t* __restrict__ db) {
  __shared__ float sum[32][65];
  __shared__ float more[4][64];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3, rows = *count;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = blockIdx.x * 64 + 8 * c;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n < width)
    for (int row = g; row < rows; row += 32) {
      float w[8];
      unpack8(*reinterpret_cast<const u32x4*>(d + row * pitch + n), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[g][8 * c + e] = v[e];
  float extra = 0.0f;
  for (int base = 64 * wave; base < rows; base += 256) {
    const int row = base + lane;
    const int t = row < rows ? tok[row] - n_first - 64 * (int)blockIdx.x : -1;
    const bool hit = (uint32_t)t < 64u;
    const float r = hit ? rest[row] : 0.0f;
    for (uint64_t hits = __ballot(hit); hits != 0; hits &= hits - 1) {
      const int from = __ffsll((unsigned long long)hits) - 1;
      const int column = __shfl(t, from, 64);
      const float value = __shfl(r, from, 64);
      if (lane == column) extra += value;
    }
  }
  more[wave][lane] = extra;
  __syncthreads();
  if (threadIdx.x < 64 && blockIdx.x * 64 + threadIdx.x < width) {
    float s = 0.0f;
    for (int i = 0; i < 32; ++i) s += sum[i][threadIdx.x];
    for (int i = 0; i < 4; ++i) s += more[i][threadIdx.x];
    db[blockIdx.x * 64 + threadIdx.x] = (uint16_t)(pack_bf16(s, 0.0f) & 0xFFFFu);
  }
}

// dz of a piece.  It bounds the workspace: 4096 x 128256 x 4096 takes 13.9 ms in pieces of 32 MB, 12.9 of 128 and 512 MB, 12.8
// of 2 GB; 16384 rows 70.8, 52.5, 51.0, 51.4 ms.
constexpr int64_t kCePieceBytes = (int64_t)128 << 20;
constexpr int64_t kCePieceMost = 1 << 18;               // its columns: 32-bit offsets

struct CeLayout {
  int64_t xc, ctok, index, count, parts, tlogit, cstats, coef, rest, hits, d, acc, bytes;
  int64_t piece, tiles;
  TileSize logits, grad;           // tiles of the two passes over the logits
  TileSplit dx;
};

// No part's size falls as M grows, though tiles, pieces and splits change with it: a workspace kept for the largest
// batch holds every smaller one.
static CeLayout ce_layout(int64_t M, int64_t V, int64_t K, bool backward) {
  CeLayout l = {};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up256(bytes);
    return here;
  };
  l.xc = take(2 * M * K);
  l.ctok = take(4 * M);
  l.index = take(4 * M);
  l.count = take(4);
  l.logits = tile_size(M, V, (K + 63) / 64, 1);
  l.tiles = (V + tile_shape(l.logits).bn - 1) / tile_shape(l.logits).bn;
  // the forward pass's part and the backward's overlap
  const int64_t common = at;
  l.parts = take(8 * M * ((V + 127) / 128));               // tiles are 128 columns at least
  l.tlogit = take(4 * M);
  if (backward) {
    const int64_t forward_end = at;
    at = common;
    l.cstats = take(8 * M);
    l.coef = take(8 * M);
    l.rest = take(4 * M);
    int64_t most = kCePieceBytes / (2 * M) / 256 * 256;
    most = most < 1024 ? 1024 : most > kCePieceMost ? kCePieceMost : most;
    const int64_t pieces = (V + most - 1) / most;
    l.piece = up256((V + pieces - 1) / pieces);
    const int64_t widest = up256(V) < kCePieceMost ? up256(V) : kCePieceMost;
    const int64_t limit = 2048 * M > kCePieceBytes ? 2048 * M : kCePieceBytes;
    const int64_t dz = 2 * M * widest < limit ? 2 * M * widest : limit;
    l.d = take(dz);
    l.hits = take(dz / (2 * 8 * kTileHitBlock) + 4 * (widest / kTileHitBlock));   // a bit for each row and block of tokens
    l.grad = tile_size(M, l.piece, (K + 63) / 64, 1);
    l.dx = tile_split(M, K, l.piece, 8, 64);
    const int64_t split = tile_split_floats(M, K, widest, 8, 64);
    l.acc = take(4 * (split > M * K ? split : M * K));
    if (at < forward_end) at = forward_end;
  }
  l.bytes = at;
  return l;
}

int64_t linear_ce_workspace_bytes(int64_t M, int64_t V, int64_t K, bool backward) {
  const int64_t b = M == 0 ? 16 : ce_layout(M, V, K, backward).bytes;
  return b < 16 ? 16 : b;
}

static TileArgs ce_logits(const void* w, int64_t V, int64_t K, const void* bias, uint8_t* ws, const CeLayout& l,
                          int64_t M) {
  TileArgs a = {};
  a.p = (const uint8_t*)w;
  a.q = ws + l.xc;
  a.p_pitch = a.q_pitch = 2 * K;
  a.p_rows = V;
  a.q_rows = M;
  a.M = (int)M;
  a.N = (int)V;
  a.K = (int)K;
  a.m_count = (const int32_t*)(ws + l.count);
  a.splits = 1;
  a.k_split = (int)((K + 63) / 64 * 64);
  a.bias = (const uint16_t*)bias;
  a.tok = (const int32_t*)(ws + l.ctok);
  return a;
}

static hipError_t launch_ce_gather(CeGather g, hipStream_t stream) {
  g.rows = 4 * ((g.M + 4095) / 4096);
  return launch_kernel((const void*)ce_gather_kernel, dim3((unsigned)((g.M + g.rows - 1) / g.rows)), dim3(256), stream,
                       g);
}

hipError_t launch_linear_ce(const void* x, int64_t M, int64_t K, const void* w, int64_t V, const void* bias,
                            const int32_t* tok, void* workspace, float* loss, float* lse, float* stats,
                            hipStream_t stream) {
  const CeLayout l = ce_layout(M, V, K, false);
  uint8_t* const ws = (uint8_t*)workspace;
  CeGather g = {};
  g.x = (const uint16_t*)x;
  g.tok = tok;
  g.M = (int)M;
  g.V = (int)V;
  g.K = (int)K;
  g.xc = (uint16_t*)(ws + l.xc);
  g.ctok = (int32_t*)(ws + l.ctok);
  g.index = (int32_t*)(ws + l.index);
  g.count = (int32_t*)(ws + l.count);
  g.loss = loss;
  g.lse = lse;
  g.stats = (float2*)stats;
  hipError_t e = launch_ce_gather(g, stream);
  if (e != hipSuccess) return e;
  TileArgs a = ce_logits(w, V, K, bias, ws, l, M);
  a.parts = (float2*)(ws + l.parts);
  a.part_pitch = (int)l.tiles;
  a.tlogit = (float*)(ws + l.tlogit);
  e = launch_tile<kTileCeStats, false, false>(a, l.logits, stream);
  if (e != hipSuccess) return e;
  return launch_kernel((const void*)ce_join_kernel, dim3((unsigned)((M + 3) / 4)), dim3(256), stream,
                       (const float2*)(ws + l.parts), (int)l.tiles, (const float*)(ws + l.tlogit),
                       (const int32_t*)g.index, (const int32_t*)g.count, loss, lse, (float2*)stats);
}

hipError_t launch_linear_ce_backward(const void* x, int64_t M, int64_t K, const void* w, int64_t V, const void* bias,
                                     const int32_t* tok, const float* stats, const float* dloss, const float* dlse,
                                     void* workspace, void* dx, void* dw, void* db, hipStream_t stream) {
  const CeLayout l = ce_layout(M, V, K, true);
  uint8_t* const ws = (uint8_t*)workspace;
  CeGather g = {};
  g.x = (const uint16_t*)x;
  g.tok = tok;
  g.M = (int)M;
  g.V = (int)V;
  g.K = (int)K;
  g.xc = (uint16_t*)(ws + l.xc);
  g.ctok = (int32_t*)(ws + l.ctok);
  g.index = (int32_t*)(ws + l.index);
  g.count = (int32_t*)(ws + l.count);
  g.stats_in = (const float2*)stats;
  g.dloss = dloss;
  g.dlse = dlse;
  g.cstats = (float2*)(ws + l.cstats);
  g.coef = (float2*)(ws + l.coef);
  g.dx = (uint16_t*)dx;
  hipError_t e = launch_ce_gather(g, stream);
  if (e != hipSuccess) return e;
  for (int64_t v0 = 0; v0 < V; v0 += l.piece) {
    const int64_t width = V - v0 < l.piece ? V - v0 : l.piece;
    const uint8_t* const wp = (const uint8_t*)w + v0 * K * 2;
    TileArgs a = ce_logits(wp, width, K, bias == nullptr ? nullptr : (const uint16_t*)bias + v0, ws, l, M);
    a.n_first = (int)v0;
    a.stats = g.cstats;
    a.coef = g.coef;
    a.rest = (float*)(ws + l.rest);
    a.hits = dw == nullptr ? nullptr : (uint32_t*)(ws + l.hits);
    a.hit_words = (int)((M + 31) / 32);
    a.out = ws + l.d;
    a.out_pitch = l.piece;
    e = launch_tile<kTileCeGrad, false, false>(a, l.grad, stream);
    if (e != hipSuccess) return e;
    if (dx != nullptr) {
      TileArgs b = {};
      b.p = wp;
      b.q = ws + l.d;
      b.p_pitch = 2 * K;
      b.q_pitch = 2 * l.piece;
      b.p_rows = width;
      b.q_rows = M;
      b.M = (int)M;
      b.N = (int)K;
      b.K = (int)width;
      b.m_count = g.count;
      b.splits = l.dx.splits;
      b.k_split = l.dx.k_split;                                   // a narrower last piece leaves the last parts empty
      b.out = ws + l.acc;
      b.out_pitch = K;
      b.accumulate = v0 > 0;
      e = launch_tile<kTileF32, true, false>(b, l.dx.size, stream);
      if (e != hipSuccess) return e;
    }
    if (dw != nullptr) {
      TileArgs b = {};
      b.p = ws + l.xc;
      b.q = ws + l.d;
      b.p_pitch = 2 * K;
      b.q_pitch = 2 * l.piece;
      b.p_rows = b.q_rows = M;
      b.M = (int)width;
      b.N = (int)K;
      b.K = (int)M;
      b.k_count = g.count;
      b.splits = 1;
      b.k_split = (int)((M + 63) / 64 * 64);
      b.out = (uint16_t*)dw + v0 * K;
      b.out_pitch = K;
      b.tok = a.tok;
      b.n_first = a.n_first;
      b.rest = a.rest;
      b.hits = a.hits;
      b.hit_words = a.hit_words;
      e = launch_tile<kTileCeWeight, true, true>(b, tile_size(width, K, (M + 63) / 64, 1, true), stream);
      if (e != hipSuccess) return e;
    }
    if (db != nullptr) {
      e = launch_kernel((const void*)ce_bias_kernel, dim3((unsigned)((width + 63) / 64)), dim3(256), stream,
                        (const uint16_t*)(ws + l.d), l.piece, (int)width, (const int32_t*)g.ctok,
                        (const float*)(ws + l.rest), (int)v0, (const int32_t*)g.count, (uint16_t*)db + v0);
      if (e != hipSuccess) return e;
    }
  }
  if (dx == nullptr) return hipSuccess;
  return launch_kernel((const void*)ce_dx_kernel, dim3((unsigned)M, (unsigned)((K + 511) / 512)), dim3(256), stream,
                       (const float*)(ws + l.acc), (int)M, (int)K, l.dx.splits, (const uint16_t*)w,
                       (const int32_t*)g.ctok, (const float*)(ws + l.rest), (const int32_t*)g.index,
                       (const int32_t*)g.count, (uint16_t*)dx);
}

}  // namespace nvfp4
