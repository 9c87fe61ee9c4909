// Dense matrix products on 128-byte slabs of the contraction (gfx950): the tile
// kernel behind the int8 product, the cross entropy and the gated block.
//
//   acc[m][n] = sum_k Q[m][k] P[n][k],   the epilogue a template parameter.
//
// Each operand is stored either with k contiguous in a row ("straight": rows n or
// m) or with k as the row ("transposed": bf16 only), so that the three products
// of a linear layer, y = x W^T, dx = dy W and dW = dy^T x, read their tensors
// as they lie.
//
// Four wavefronts, WN x WM of them over the tile, each IT x JT tiles of
// v_mfma_f32_32x32x16_bf16 (or v_mfma_i32_32x32x32_i8: the same bytes).  The n side is
// the instruction's row operand, so that a lane's accumulators are runs of four
// n of one m.  A step is 128 bytes of k (64 bf16, 128 int8) in four sub-steps.
//
// Copies go straight to LDS (buffer loads with the LDS flag; what lies past an
// operand's end reads as zero), spread evenly over the MFMAs (all of a step's in one
// sub-step overfill the memory pipe and hold the MFMAs back: 4096 x 28672 x 4096 900 us, 750 spread).
// One barrier a step.  Two schedules:
//   * units (tiles of 256 x 256, 192 x 256 and two of 128 x 128 a compute unit): LDS holds five half
//     steps P, Q, P, Q, P.  Fragments are read a sub-step ahead.  Before sub-step 3 a wavefront waits for
//     the next step's copies, the barrier frees both halves of this one, and until the next barrier the
//     copies of Q two steps on and of P three steps on take their places;
//   * whole steps (tiles of few rows): a ring of R steps, fragments read a whole step ahead, since
//     a sub-step of two or four MFMAs is shorter than an LDS read takes.
// Straight rows take 128 bytes of LDS, their 16-byte pieces swizzled by the row;
// half h of the wavefront supplies pieces 4 h + u in sub-step u.  A transposed
// tile keeps its rows of k; ds_read_b64_tr_b16 hands each lane four k of one
// column, twice for the eight k of a fragment, in the same order of k.
//
// What bounds it.  Large products: the card's power.  With the matrix units 66 to 82 % busy
// the clock falls to 1.3 to 1.5 GHz (1.2 to 1.38 PFLOP/s, int8 2.3 POPS; a library product reaches 1.18 to
// 1.47 and 2.5; the same products of zeros run 1.4 times as fast).  Few rows: HBM, 5.2 to 5.7 TB/s.  Between, from 65 to
// some 500 rows: rows of padding, starts and epilogues of one or two rounds of workgroups.  Few columns too: the compute units
// without a tile, where K is not split.  The 256 x 256 forms with the softmax's sums, the gate and the scales spill 34,
// 16 and 4 registers a lane around their epilogues, none in the steps (the sums of 3890 x 128256 write 290 MB for it).
#pragma once

#include <type_traits>

#include "nvfp4_device.hpp"
#include "nvfp4_launch.hpp"

namespace nvfp4 {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2t __attribute__((ext_vector_type(2)));

enum TileEpilogue : int {
  kTileBf16,        // out bf16 [m][n]
  kTileF32,         // out float [split][m][n], added to what is there if accumulate
  kTileInt8,        // out bf16 [m][n] = acc * sx[m] * sw[n] + bias[n]
  kTileGated,       // P = [gate; up]: out a = silu(g) u, optionally h = [g, u] in float32
  kTileGatedBack,   // acc = da: dh = [da u silu'(g), da silu(g)], from h
  kTileCeStats,     // per (m, tile of n): maximum and sum of exp, and the target's logit
  kTileCeGrad,      // out bf16 [m][n] = gradient of the logits
  kTileCeWeight     // out bf16 [m][n], m a token: acc + sum over the rows i with that target of bf16(rest[i]) * P[i][n]
};

struct TileArgs {
  const uint8_t* p;          // n side
  const uint8_t* q;          // m side
  int64_t p_pitch, q_pitch;  // bytes of a stored row
  int64_t p_rows, q_rows;    // rows stored (straight: rows of the side; transposed: rows of k)
  int32_t M, N, K;           // K in elements, a multiple of a 16-byte piece
  const int32_t* m_count;    // device count in place of M, q_rows (NULL: none)
  const int32_t* k_count;    // device count in place of K, p_rows and q_rows (transposed sides)
  int32_t m_tiles, n_tiles, splits, k_split;   // k of a split, a multiple of a step
  void* out;
  int64_t out_pitch;         // elements
  int32_t accumulate;
  int32_t turn_by_tile;      // the launcher's: where a workgroup starts in K
  // epilogues
  const float* sx;
  const float* sw;
  const uint16_t* bias;      // [n]
  int32_t I;                 // gated: width of a half
  int32_t pair_rows;         // where not 0: gated, out row pair_rows + m receives what rounding took from row m; float32,
                             // row pair_rows + m of the product is added to row m (M = 2 pair_rows, within one pass)
  uint16_t* act;             // gated: the rounded a once more [m][I], or NULL
  float* h;                  // gated: [m][2 I], written (forward, may be NULL) or read (backward)
  uint16_t* dh;              // gated backward [m][2 I]
  const int32_t* tok;        // [m] target of each row
  float2* parts;             // [m][part_pitch]
  int32_t part_pitch, n_first;   // n_first: n of column 0 (a piece of the vocabulary)
  float* tlogit;             // [m]
  const float2* stats;       // [m] (maximum, sum)
  const float2* coef;        // [m] (dloss + dlse, dloss)
  float* rest;               // [row] what rounding took from the gradient of the target's logit
  uint32_t* hits;            // [block of kTileHitBlock tokens][hit_words] bits of the rows whose target is in the block:
                             // written by the gradient of the logits (may be NULL), read by the weight's
  int32_t hit_words;
};
constexpr int kTileHitBlock = 128;

// s_waitcnt immediate: vmcnt(vm) lgkmcnt(0), expcnt left alone
constexpr int tile_wait(int vm) { return (vm & 15) | ((vm >> 4) << 14) | 0x0070; }
constexpr int kTileThreads = 256;
constexpr uint32_t kTileNowhere = 0xF0000000u;   // a buffer offset past every operand: reads as zero

typedef __attribute__((address_space(3))) void* tile_lds_t;
typedef __attribute__((address_space(3))) s16x4* tile_tr_t;

// A transposing LDS read.  __restrict gives the read alias information: without any, the compiler waits before
// it for every copy to LDS in flight, as it does not for ordinary LDS reads.
__device__ __forceinline__ s16x4 tile_read_tr(tile_tr_t __restrict at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(at);
}

__device__ __forceinline__ void tile_copy16(__amdgpu_buffer_rsrc_t r, tile_lds_t dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, voff, soff, 0, 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {      // nearest even; NaN stays NaN
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2t));
}
// What rounding v to hi left over; nothing where hi is not finite (an infinity's product or sum is the one of hi alone).
__device__ __forceinline__ float rest_bf16(float v, float hi) { return fabsf(hi) < INFINITY ? v - hi : 0.0f; }
// A remainder's product: with an infinite factor the result is the one of the rounded value alone, the remainder's
// being infinite of either sign, or NaN where it is 0.
__device__ __forceinline__ float finite_or_0(float v) { return fabsf(v) < INFINITY ? v : 0.0f; }
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void unpack8(u32x4 w, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = bf16_lo(w[e]);
    v[2 * e + 1] = bf16_hi(w[e]);
  }
}
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }
__device__ __forceinline__ float sigmoid_fast(float g) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-g)); }

template <int IT_, int JT_, int WN_, int WM_, bool PT_, bool QT_, int EPI_, int R_>
struct TileCfg {
  static constexpr int IT = IT_, JT = JT_, WN = WN_, WM = WM_, EPI = EPI_, R = R_;
  static constexpr bool PT = PT_, QT = QT_, I8 = EPI_ == kTileInt8;
  static constexpr int BN = 32 * IT * WN, BM = 32 * JT * WM;
  static constexpr int KE = I8 ? 128 : 64;                      // elements of k per step
  static constexpr int kPBytes = BN * 128, kQBytes = BM * 128;
  // R = 0: five units of half a step (P, Q, P, Q, P ...); else R whole steps
  static constexpr bool kUnits = R == 0;
  static constexpr int kBuf = kPBytes + kQBytes;
  static constexpr int kRing = kUnits ? 5 : R;                  // steps until a buffer returns to its place
  static constexpr int kCopies = kBuf / 4096;                   // copies per wavefront per step
  static constexpr int copy_slot(int c) { return (8 * c + 1) * 2 * IT * JT / (4 * kCopies); }   // even spacing
  static constexpr int kRingBytes = kUnits ? 5 * kPBytes : R * kBuf;
  static constexpr int p_at(int ph) { return kUnits ? 2 * ph % 5 * kPBytes : ph * kBuf; }
  static constexpr int q_at(int ph) { return kUnits ? (2 * ph + 1) % 5 * kPBytes : ph * kBuf + kPBytes; }
  // epilogue: rows in float32, 32 of each wavefront at a time, or bf16 outputs, all of them (gated: 32, with g and u
  // in float32 before them)
  static constexpr bool kStageF32 = EPI == kTileF32 || EPI == kTileGatedBack;
  static constexpr int kStageRows = 32 * WM, kStagePitch = BN + 4;
  static constexpr int kStageJ = EPI == kTileGated ? 1 : JT;
  static constexpr int kOutPitch = (EPI == kTileGated ? BN / 2 * 6 : BN) + 8;   // in bf16
  static constexpr int kStage = kStageF32 ? kStageRows * kStagePitch * 4 : 32 * kStageJ * WM * kOutPitch * 2;
  static constexpr int kLds = kRingBytes > kStage ? kRingBytes : kStage;
  static constexpr int kPerCu = kLds <= 80 * 1024 ? 2 : 1;      // workgroups meant to share a compute unit
  static_assert(WN * WM == 4 && kLds <= 160 * 1024, "tile");
  static_assert(!I8 || (!PT && !QT), "int8 operands are straight");
  static_assert((!PT || 512 % BN == 0) && (!QT || 512 % BM == 0), "a copy fills whole rows of a transposed tile");
  static_assert(kUnits ? BN >= BM : R >= 2 && R <= 4 && R * kCopies < 64, "ring");
};

template <class C>
__global__ __launch_bounds__(kTileThreads, C::kPerCu) void dense_tile_kernel(TileArgs a) {
  constexpr int IT = C::IT, JT = C::JT, R = C::R, BN = C::BN, BM = C::BM;
  constexpr bool PT = C::PT, QT = C::QT;
  constexpr int kPC = BN / 32, kQC = BM / 32;                    // copies of each side
  constexpr int kMf = IT * JT;                                  // MFMAs per sub-step
  constexpr int kReads = IT * (PT ? 2 : 1) + JT * (QT ? 2 : 1);
  using Acc = std::conditional_t<C::I8, i32x16, f32x16>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % C::WN, wm = wave / C::WN;
  const int r = lane & 31, h = lane >> 5;

  // Workgroup b runs on XCD b % 8: each XCD takes one run of tiles, and in it
  // patches of up to eight tiles of m under neighbouring tiles of n, so that
  // what its compute units copy at a time meets in its own L2.
  const int total = gridDim.x, xcd = blockIdx.x & 7;
  const int t = xcd * (total >> 3) + min(xcd, total & 7) + (blockIdx.x >> 3);
  const int tiles = a.m_tiles * a.n_tiles;
  const int split = t / tiles, tile = t % tiles;
  const int group = tile / (8 * a.n_tiles), in_group = tile % (8 * a.n_tiles);
  const int gm = min(8, a.m_tiles - 8 * group);
  const int m0 = (8 * group + in_group % gm) * BM, nt = in_group / gm;
  const int n0 = nt * (C::EPI == kTileGated ? BN / 2 : BN);
  const int M = a.m_count ? *a.m_count : a.M;
  if (m0 >= M) return;
  const int K = a.k_count ? *a.k_count : a.K;
  const int k_begin = split * a.k_split, k_end = min(K, k_begin + a.k_split);
  const int nsteps = k_end > k_begin ? (k_end - k_begin + C::KE - 1) / C::KE : 0;

  // Straight rows a power of two apart put one step of every row on few memory channels, and workgroups that start
  // together would all be at that step: they start at different ones (one token, 128256 x 4096 int8: 110 -> 94 us).
  // Rows of k are read whole by neighbouring tiles, which should stay together (dx of 4096 x 28672 x 4096: 700 -> 820 us).
  const int turn = PT || nsteps == 0 ? 0 : a.turn_by_tile ? nt % nsteps : (xcd * nsteps) >> 3;

  // Straight copies: instruction c of wavefront w fills rows 8 (4 c + w) .. + 7, lane l slot l & 7 of row
  // 8 (4 c + w) + (l >> 3), i.e. piece (l & 7) ^ (l >> 3) ^ (w & 1).  Transposed: with W columns a
  // row has W / 8 pieces; lane l fills slot l % (W / 8) of row l / (W / 8) of the instruction's.
  const int piece = (lane & 7) ^ (lane >> 3) ^ (wave & 1);
  const uint8_t* p_base;
  const uint8_t* q_base;
  uint32_t p_range = 0, q_range = 0, p_off, q_off;
  constexpr int kPPr = BN / 8, kQPr = BM / 8;                   // pieces of a transposed row
  auto tr_swizzle = [](int row, int pieces) { return pieces >= 16 ? 4 * (row & 3) : 0; };
  if (!PT) {
    p_base = a.p + (int64_t)n0 * a.p_pitch;
    p_range = (uint32_t)min((int64_t)0xE0000000u, (a.p_rows - n0) * a.p_pitch);
    p_off = (uint32_t)((8 * wave + (lane >> 3)) * a.p_pitch + 16 * piece);
  } else {
    p_base = a.p + (int64_t)n0 * 2;
    const int row = wave * (64 / kPPr) + lane / kPPr;
    p_off = (uint32_t)(row * a.p_pitch + 16 * ((lane % kPPr) ^ tr_swizzle(row, kPPr)));
  }
  if (!QT) {
    q_base = a.q + (int64_t)m0 * a.q_pitch;
    q_range = (uint32_t)min((int64_t)0xE0000000u, ((a.m_count ? M : a.q_rows) - m0) * a.q_pitch);
    q_off = (uint32_t)((8 * wave + (lane >> 3)) * a.q_pitch + 16 * piece);
  } else {
    q_base = a.q + (int64_t)m0 * 2;
    const int row = wave * (64 / kQPr) + lane / kQPr;
    q_off = (uint32_t)(row * a.q_pitch + 16 * ((lane % kQPr) ^ tr_swizzle(row, kQPr)));
  }
  const int piece_k = piece * (C::KE / 8);
  // row of P's tile at which copy c starts, relative to n0 (gated: each wavefront column's rows are its
  // gates, then its ups)
  auto p_row = [&](int c) __attribute__((always_inline)) -> int64_t {
    if constexpr (C::EPI == kTileGated) {
      constexpr int half = 16 * IT;
      const int row = 32 * c, g = row / (2 * half), in = row % (2 * half);
      return in < half ? half * g + in : (int64_t)a.I + half * g + in - half;
    } else {
      return 32 * c;
    }
  };

  // copy c of step st into ring buffer ph (steps past the last: nothing is read, zeros arrive)
  auto copy_one = [&](int st, int ph, int c) __attribute__((always_inline)) {
    const bool live = st < nsteps;
    const int turned = st + turn;
    const int k0 = k_begin + (turned < nsteps ? turned : turned - nsteps) * C::KE;
    const bool left = c < kPC;
    const int i = left ? c : c - kPC;
    uint8_t* const dst = lds + (left ? C::p_at(ph) : C::q_at(ph)) + (4 * i + wave) * 1024;
    const int64_t pitch = left ? a.p_pitch : a.q_pitch;
    if (left ? !PT : !QT) {
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(left ? p_base : q_base), (short)0, live ? (int)(left ? p_range : q_range) : 0, 0x00020000);
      const uint32_t off = (left ? p_off : q_off) + (uint32_t)((left ? p_row(i) : 32 * i) * pitch);
      tile_copy16(rs, (tile_lds_t)dst, k0 + piece_k < K ? off : kTileNowhere, live ? k0 * (128 / C::KE) : 0);
    } else {
      const int rows = live ? min(K - k0, 64) : 0;               // no branch: the loop stays one block
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void*)((left ? p_base : q_base) + k0 * pitch), (short)0,
                                            max(rows * (int)pitch - 2 * (left ? n0 : m0), 0), 0x00020000);
      tile_copy16(rs, (tile_lds_t)dst, (left ? p_off : q_off) + (uint32_t)(i * (256 / (left ? kPPr : kQPr)) * pitch), 0);
    }
  };

  // Fragment reads.  Straight: row 32 i + r of the wavefront's, piece 4 h + u.  Transposed: lane l of a
  // group of 16 names row k = l / 4 and columns 4 (l % 4) .. + 3 and receives column l's four k.
  const int sw = (r & 7) ^ ((r >> 3) & 1);
  const int l16 = lane & 15, k4 = l16 >> 2;
  auto tr_lane = [&](int pieces, int tile0) __attribute__((always_inline)) {   // XORed with 64 i for 32-column tile i
    return (uint32_t)((32 * h + k4) * pieces * 16 + 64 * (tile0 ^ (pieces >= 16 ? k4 : 0)) + 32 * ((lane >> 4) & 1) +
                      8 * (l16 & 3));
  };
  uint32_t tr_p = PT ? tr_lane(kPPr, IT * wn) : 0, tr_q = QT ? tr_lane(kQPr, JT * wm) : 0;
  auto frag_straight = [&](const uint8_t* base, int row0, int u) __attribute__((always_inline)) {
    return *reinterpret_cast<const u32x4*>(base + (row0 + r) * 128 + 16 * ((4 * h + u) ^ sw));
  };
  auto frag_tr = [&](const uint8_t* base, uint32_t at, int pieces, int i, int u, int e) __attribute__((always_inline)) {
    return __builtin_bit_cast(uint2, tile_read_tr((tile_tr_t)(base + (at ^ (64 * i)) + (8 * u + 4 * e) * pieces * 16)));
  };
  // fragments: two sub-steps' (units), or two steps'
  constexpr int kSets = C::kUnits ? 2 : 8;
  u32x4 pf[kSets][IT], qf[kSets][JT];
  auto read_one = [&](int ph, int u, int x, u32x4 (&pn)[IT], u32x4 (&qn)[JT]) __attribute__((always_inline)) {
    const uint8_t* const pb = lds + C::p_at(ph);
    constexpr int np = IT * (PT ? 2 : 1);
    if (x < np) {
      if constexpr (!PT) {
        pn[x] = frag_straight(pb, 32 * IT * wn + 32 * x, u);
      } else {
        const uint2 v = frag_tr(pb, tr_p, kPPr, x / 2, u, x % 2);
        pn[x / 2][2 * (x % 2)] = v.x;
        pn[x / 2][2 * (x % 2) + 1] = v.y;
      }
    } else {
      const int y = x - np;
      const uint8_t* const qb = lds + C::q_at(ph);
      if constexpr (!QT) {
        qn[y] = frag_straight(qb, 32 * JT * wm + 32 * y, u);
      } else {
        const uint2 v = frag_tr(qb, tr_q, kQPr, y / 2, u, y % 2);
        qn[y / 2][2 * (y % 2)] = v.x;
        qn[y / 2][2 * (y % 2) + 1] = v.y;
      }
    }
  };

  Acc acc[IT][JT];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;

  auto mfma = [&](u32x4 p, u32x4 q, Acc c) __attribute__((always_inline)) {
    if constexpr (C::I8)
      return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, p), __builtin_bit_cast(i32x4, q), c, 0, 0,
                                                   0);
    else
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c,
                                                     0, 0, 0);
  };

  // Units: copies after MFMA s of sub-step u of step st (ring place ph), spread evenly between two barriers: Q of
  // the step after next, then P of the step behind it.
  auto copy_slot = [&](int st, auto PH, int u, int s) __attribute__((always_inline)) {
    constexpr int ph = decltype(PH)::value;
    const int ahead = u == 3 ? 1 : 0;                           // the period belongs to the step of its barrier
#pragma unroll
    for (int c = 0; c < C::kCopies; ++c) {
      if (((u + 1) & 3) * kMf + s != C::copy_slot(c)) continue;  // slots counted from the barrier on
      if (c < kQC) copy_one(st + ahead + 1, (ph + ahead + 1) % 5, kPC + c);
      else copy_one(st + ahead + 2, (ph + ahead + 2) % 5, c - kQC);
    }
  };
  auto kstep = [&](int st, auto PH, auto ODD) __attribute__((always_inline)) {
    constexpr int ph = decltype(PH)::value, ph1 = (ph + 1) % C::kRing;
    if constexpr (C::kUnits) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u == 3) {
          __builtin_amdgcn_s_waitcnt(tile_wait(kPC));
          asm volatile("s_barrier" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
        }
        u32x4(&pc)[IT] = pf[u & 1];
        u32x4(&qc)[JT] = qf[u & 1];
#pragma unroll
        for (int s = 0; s < kMf; ++s) {
          acc[s / JT][s % JT] = mfma(pc[s / JT], qc[s % JT], acc[s / JT][s % JT]);
#pragma unroll
          for (int x = 0; x < kReads; ++x)
            if (x * kMf / kReads == s) read_one(u < 3 ? ph : ph1, (u + 1) & 3, x, pf[(u + 1) & 1], qf[(u + 1) & 1]);
          copy_slot(st, PH, u, s);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
      constexpr int now = 4 * decltype(ODD)::value, next = 4 - now;
      __builtin_amdgcn_s_waitcnt(tile_wait((R - 2) * C::kCopies));   // step st + 1 has landed, this wavefront has read step st
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < 4 * kMf; ++t) {
        const int u = t / kMf, s = t % kMf;
        acc[s / JT][s % JT] = mfma(pf[now + u][s / JT], qf[now + u][s % JT], acc[s / JT][s % JT]);
#pragma unroll
        for (int x = 0; x < 4 * kReads; ++x)
          if (x * kMf / kReads == t) read_one(ph1, x / kReads, x % kReads, pf[next + x / kReads], qf[next + x / kReads]);
#pragma unroll
        for (int c = 0; c < C::kCopies; ++c)
          if (c * 4 * kMf / C::kCopies == t) copy_one(st + R, ph, c);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // kTileCeWeight: bits of the rows 32 word .. + 31 that have their target in this tile, the first ones under way early
  constexpr int kHitBlocks = C::EPI == kTileCeWeight ? BM / kTileHitBlock : 1;
  const int hit_words = C::EPI == kTileCeWeight ? (K + 31) / 32 : 0;
  uint32_t hit[kHitBlocks] = {};
  auto read_hits = [&](int word) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < kHitBlocks; ++b)
      hit[b] = word < hit_words && m0 + kTileHitBlock * b < M
                   ? a.hits[(int64_t)(m0 / kTileHitBlock + b) * a.hit_words + word] : 0u;
  };
  if constexpr (C::EPI == kTileCeWeight) read_hits(tid);

  if constexpr (C::kUnits) {
    constexpr int early = (C::kCopies + 3) / 4;                 // what sub-step 3 before the first would have copied
    static_assert(C::copy_slot(early - 1) < kMf && C::copy_slot(early) >= kMf && early <= kQC, "copies before sub-step 0");
#pragma unroll
    for (int x = 0; x < C::kCopies + kPC; ++x) copy_one(x / C::kCopies, x / C::kCopies, x % C::kCopies);
#pragma unroll
    for (int x = 0; x < early; ++x) copy_one(1, 1, kPC + x);
    __builtin_amdgcn_s_waitcnt(tile_wait(kPC + early));
  } else {
#pragma unroll
    for (int x = 0; x < R * C::kCopies; ++x) copy_one(x / C::kCopies, x / C::kCopies, x % C::kCopies);
    __builtin_amdgcn_s_waitcnt(tile_wait((R - 1) * C::kCopies));
  }
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int x = 0; x < (C::kUnits ? 1 : 4) * kReads; ++x)
    read_one(0, x / kReads, x % kReads, pf[x / kReads], qf[x / kReads]);

  int st = 0;
  using std::integral_constant;
  // a loop's length: places of the ring, and for whole steps both halves of the fragment registers
  constexpr int kLoop = !C::kUnits && C::kRing % 2 ? 2 * C::kRing : C::kRing;
  auto step = [&](auto X) __attribute__((always_inline)) {
    constexpr int x = decltype(X)::value;
    kstep(st + x, integral_constant<int, x % C::kRing>{}, integral_constant<int, x % 2>{});
  };
  auto rest = [&](auto X) __attribute__((always_inline)) {
    constexpr int x = decltype(X)::value;
    if constexpr (x < kLoop - 1)
      if (st + x < nsteps) step(X);
  };
  for (; st + kLoop <= nsteps; st += kLoop) {
    step(integral_constant<int, 0>{});
    step(integral_constant<int, 1>{});
    if constexpr (kLoop > 2) step(integral_constant<int, 2>{});
    if constexpr (kLoop > 3) step(integral_constant<int, 3>{});
    if constexpr (kLoop > 4) step(integral_constant<int, 4>{});
    if constexpr (kLoop > 5) step(integral_constant<int, 5>{});
  }
  static_assert(kLoop <= 6, "steps of the loop");
  rest(integral_constant<int, 0>{});
  rest(integral_constant<int, 1>{});
  rest(integral_constant<int, 2>{});
  rest(integral_constant<int, 3>{});
  rest(integral_constant<int, 4>{});
  __builtin_amdgcn_s_waitcnt(tile_wait(0));
  __syncthreads();

  if constexpr (C::EPI == kTileCeWeight) {
    // The remainders, as steps of their own: the rows that have their target in this tile, in order, 64 at a time, P of
    // them against one remainder each, rounded to bf16.  Few tiles have any: of 4096 rows 8 have their target among 256
    // of 128256 tokens.  Rows lie so that a sub-step takes 16 of them (step of 333 x 32003 x 2080: 253 us; with
    // four sub-steps always 265, without the remainders 243).
    static_assert(C::kUnits && PT && QT && BM % kTileHitBlock == 0, "remainders");
    constexpr int kEnd = kPPr * 1024 + kQPr * 1024;              // of a step's P and Q
    uint8_t* const pb = lds + C::p_at(0);
    uint8_t* const qb = lds + C::q_at(0);
    static_assert(C::p_at(0) == 0 && C::q_at(0) == C::kPBytes && kEnd + 512 <= C::kLds, "remainders");
    int* const from = reinterpret_cast<int*>(lds + kEnd);
    int* const part = from + 64;
    for (int base = 0; base < hit_words; base += kTileThreads) {
      const int word = base + tid;
      if (base > 0) read_hits(word);
      uint32_t bits = 0;
#pragma unroll
      for (int b = 0; b < kHitBlocks; ++b) bits |= hit[b];
      int sum = __popc(bits);                                    // up to and with this thread's
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int below = __shfl_up(sum, d, 64);
        sum += lane >= d ? below : 0;
      }
      if (lane == 63) part[wave] = sum;
      __syncthreads();
      int first = sum - __popc(bits), total = 0;
#pragma unroll
      for (int w = 0; w < kTileThreads / 64; ++w) {
        first += w < wave ? part[w] : 0;
        total += part[w];
      }
      for (int done = 0; done < total; done += 64) {
        const int count = min(total - done, 64);
        int at = first - done;
        for (uint32_t left = bits; left != 0; left &= left - 1, ++at)
          if ((uint32_t)at < 64u) from[at] = 32 * word + __ffs((int)left) - 1;
        const int steps = (count + 15) / 16;                     // sub-steps, 16 rows each
        auto place = [&](int x) __attribute__((always_inline)) { return 8 * (x >> 4) + 32 * ((x >> 3) & 1) + (x & 7); };
        for (int e = tid; e < 16 * steps * kQPr; e += kTileThreads)
          *reinterpret_cast<u32x4*>(qb + 16 * (place(e / kQPr) * kQPr + e % kQPr)) = u32x4{0, 0, 0, 0};
        __syncthreads();
        if (tid < count) {
          const int i = from[tid], m = a.tok[i] - a.n_first - m0, k = place(tid);
          *reinterpret_cast<uint16_t*>(qb + 16 * (k * kQPr + ((m >> 3) ^ tr_swizzle(k, kQPr))) + 2 * (m & 7)) =
              (uint16_t)pack_bf16(a.rest[i], 0.0f);
        }
        for (int e = tid; e < 16 * steps * kPPr; e += kTileThreads) {
          const int x = e / kPPr, k = place(x), n = n0 + 8 * (e % kPPr ^ tr_swizzle(k, kPPr));
          u32x4 v = {0, 0, 0, 0};
          if (x < count && n < a.N) v = *reinterpret_cast<const u32x4*>(a.p + from[x] * a.p_pitch + 2 * n);
          *reinterpret_cast<u32x4*>(pb + 16 * (k * kPPr + e % kPPr)) = v;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (u >= steps) break;
#pragma unroll
          for (int x = 0; x < kReads; ++x) read_one(0, u, x, pf[u & 1], qf[u & 1]);
#pragma unroll
          for (int s = 0; s < kMf; ++s) acc[s / JT][s % JT] = mfma(pf[u & 1][s / JT], qf[u & 1][s % JT], acc[s / JT][s % JT]);
        }
        __syncthreads();                                         // before the next ones take their places
      }
      if (total == 0) __syncthreads();                           // part is read before it is written again
    }
  }
  if constexpr (C::EPI == kTileCeStats) {
    // Each lane holds 16 IT logits of each of its JT rows; wavefronts of a row meet in LDS.
    float2* const red = reinterpret_cast<float2*>(lds);          // [WN][BM]
    const int nb = n0 + 32 * IT * wn + 4 * h;                    // accumulator 4 q + v of row tile i: n = nb + 32 i + 8 q + v
    if (a.bias != nullptr || n0 + BN > a.N) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int n = nb + 32 * i + 8 * q + v;
            const float b =
                n >= a.N ? -INFINITY : a.bias != nullptr ? __uint_as_float((uint32_t)a.bias[n] << 16) : 0.0f;
#pragma unroll
            for (int j = 0; j < JT; ++j)
              acc[i][j][4 * q + v] = n >= a.N ? -INFINITY : acc[i][j][4 * q + v] + b;
          }
    }
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      const int ml = 32 * (JT * wm + j) + r, m = m0 + ml;
      const int tok = m < M ? a.tok[m] - a.n_first - nb : -1;
      float mx = -INFINITY, s = 0.0f, zt = 0.0f;
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          mx = fmaxf(mx, acc[i][j][v]);
          zt = tok == 32 * i + 8 * (v >> 2) + (v & 3) ? acc[i][j][v] : zt;
        }
      if (tok >= 0 && tok < 32 * IT && (tok & 4) == 0) a.tlogit[m] = zt;
      // halves of a row in two lanes: one maximum for both
      const float mm = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float ref = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) s += exp_fast(acc[i][j][v] - ref);
      s += __shfl_xor(s, 32, 64);
      if (h == 0) red[wn * BM + ml] = make_float2(mm, s);
    }
    __syncthreads();
    for (int ml = tid; ml < BM; ml += kTileThreads) {
      if (m0 + ml >= M) continue;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::WN; ++w) mm = fmaxf(mm, red[w * BM + ml].x);
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < C::WN; ++w) {
        const float2 v = red[w * BM + ml];
        s += v.x == -INFINITY ? v.y : v.y * exp_fast(v.x - mm);    // -inf: no logit, 0, or NaN
      }
      a.parts[(int64_t)(m0 + ml) * a.part_pitch + nt] = make_float2(mm, s);
    }
    return;
  } else if constexpr (C::kStageF32) {
    // 32 rows of each wavefront row at a time through LDS in float32, so that memory is read and written in
    // whole lines; a pass's reads are under way before its rows are in place.
    float* const stage = reinterpret_cast<float*>(lds);
    constexpr int kChunks = BN / 8, kIters = C::kStageRows * kChunks / kTileThreads;
    const int c = tid % kChunks, n = n0 + 8 * c;
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      f32x4 in[kIters][C::EPI == kTileF32 ? 2 : 4];
      int64_t at[kIters];
      bool on[kIters];
#pragma unroll
      for (int it = 0; it < kIters; ++it) {
        const int row = tid / kChunks + it * (kTileThreads / kChunks);
        const int m = m0 + 32 * (JT * (row >> 5) + j) + (row & 31);
        on[it] = m < M && n < a.N;
        if constexpr (C::EPI == kTileF32) {
          if (a.pair_rows != 0) on[it] = on[it] && m < a.pair_rows;
          at[it] = ((int64_t)split * (a.pair_rows != 0 ? a.pair_rows : a.M) + m) * a.out_pitch + n;
          if (on[it] && a.accumulate) {
            in[it][0] = *reinterpret_cast<const f32x4*>((const float*)a.out + at[it]);
            in[it][1] = *reinterpret_cast<const f32x4*>((const float*)a.out + at[it] + 4);
          }
        } else {
          at[it] = m;
          if (on[it]) {
            const float* const hp = a.h + (int64_t)m * 2 * a.I + n;
            in[it][0] = *reinterpret_cast<const f32x4*>(hp);
            in[it][1] = *reinterpret_cast<const f32x4*>(hp + 4);
            in[it][2] = *reinterpret_cast<const f32x4*>(hp + a.I);
            in[it][3] = *reinterpret_cast<const f32x4*>(hp + a.I + 4);
          }
        }
      }
      if (j > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
          *reinterpret_cast<f32x4*>(stage + (32 * wm + r) * C::kStagePitch + 32 * (IT * wn + i) + 8 * q + 4 * h) = v;
        }
      __syncthreads();
#pragma unroll
      for (int it = 0; it < kIters; ++it) {
        const int row = tid / kChunks + it * (kTileThreads / kChunks);
        const f32x4* const src = reinterpret_cast<const f32x4*>(stage + row * C::kStagePitch + 8 * c);
        f32x4 lo = src[0], hi = src[1];
        if (!on[it]) continue;
        if constexpr (C::EPI == kTileF32) {
          if (a.pair_rows != 0) {
            const f32x4* const low = reinterpret_cast<const f32x4*>(stage + (row + a.pair_rows) * C::kStagePitch + 8 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              lo[e] += finite_or_0(low[0][e]);
              hi[e] += finite_or_0(low[1][e]);
            }
          }
          if (a.accumulate) {
            lo += in[it][0];
            hi += in[it][1];
          }
          *reinterpret_cast<f32x4*>((float*)a.out + at[it]) = lo;
          *reinterpret_cast<f32x4*>((float*)a.out + at[it] + 4) = hi;
        } else {
          float dg[8], du[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = e < 4 ? lo[e & 3] : hi[e & 3], g = in[it][e >> 2][e & 3], u = in[it][2 + (e >> 2)][e & 3];
            const float s = sigmoid_fast(g), gs = g * s;
            du[e] = v * gs;
            dg[e] = v * u * (s + gs * (1.0f - s));
          }
          *reinterpret_cast<u32x4*>(a.dh + at[it] * 2 * a.I + n) = pack8(dg);
          *reinterpret_cast<u32x4*>(a.dh + at[it] * 2 * a.I + a.I + n) = pack8(du);
        }
      }
    }
  } else {
    // Outputs are made in registers, rounded, and gathered in LDS so that memory is written in whole lines.
    constexpr int kW = C::EPI == kTileGated ? BN / 2 : BN;       // columns written
    constexpr int kJP = C::kStageJ;                              // column tiles of a wavefront per pass
    uint16_t* const stage = reinterpret_cast<uint16_t*>(lds);
    if constexpr (C::EPI == kTileCeGrad) {
      const int m = m0 + tid, t = tid < BM && m < M ? a.tok[m] - a.n_first - n0 : -1;
      if (a.hits != nullptr && 64 * wave < BM) {
#pragma unroll
        for (int b = 0; b < BN / kTileHitBlock; ++b) {
          const uint64_t bits = __ballot(t >= 0 && t / kTileHitBlock == b);
          const int word = m0 / 32 + 2 * wave + h;
          if (r == 0 && 32 * (2 * wave + h) < BM && word < a.hit_words)
            a.hits[(int64_t)(n0 / kTileHitBlock + b) * a.hit_words + word] = (uint32_t)(bits >> (32 * h));
        }
      }
    }
    float cs[C::I8 ? IT : 1][4][4], cb[C::I8 || C::EPI == kTileCeGrad ? IT : 1][4][4];
    const bool has_bias = (C::I8 || C::EPI == kTileCeGrad) && a.bias != nullptr;
    if constexpr (C::I8 || C::EPI == kTileCeGrad) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + 32 * (IT * wn + i) + 8 * q + 4 * h;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int ne = min(n + e, a.N - 1);
            if constexpr (C::I8) cs[i][q][e] = a.sw[ne];
            cb[i][q][e] = has_bias ? __uint_as_float((uint32_t)a.bias[ne] << 16) : 0.0f;
          }
        }
    }
#pragma unroll
    for (int j0 = 0; j0 < JT; j0 += kJP) {
      if (j0 > 0) __syncthreads();
#pragma unroll
      for (int jj = 0; jj < kJP; ++jj) {
        const int j = j0 + jj, m = m0 + 32 * (JT * wm + j) + r;
        uint16_t* const to = stage + (32 * (kJP * wm + jj) + r) * C::kOutPitch;
        if constexpr (C::EPI == kTileGated) {
#pragma unroll
          for (int i = 0; i < IT / 2; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int at = 32 * (IT / 2 * wn + i) + 8 * q + 4 * h;
              f32x4 g, u;
              float o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                g[e] = acc[i][j][4 * q + e];
                u[e] = acc[i + IT / 2][j][4 * q + e];
                o[e] = g[e] * sigmoid_fast(g[e]) * u[e];
              }
              const uint2 hi = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
              *reinterpret_cast<uint2*>(to + 4 * kW + at) = hi;
              if (a.pair_rows != 0)
                *reinterpret_cast<uint2*>(to + 5 * kW + at) =
                    make_uint2(pack_bf16(rest_bf16(o[0], bf16_lo(hi.x)), rest_bf16(o[1], bf16_hi(hi.x))),
                               pack_bf16(rest_bf16(o[2], bf16_lo(hi.y)), rest_bf16(o[3], bf16_hi(hi.y))));
              if (a.h != nullptr) {
                *reinterpret_cast<f32x4*>((float*)to + at) = g;
                *reinterpret_cast<f32x4*>((float*)to + kW + at) = u;
              }
            }
        } else {
          float sx = 1.0f, top = 0.0f, scale = 0.0f, minus = 0.0f, at_target = 0.0f;
          int tok = -1;
          if constexpr (C::I8) sx = a.sx[min(m, M - 1)];
          if constexpr (C::EPI == kTileCeGrad) {
            const int mc = min(m, M - 1);
            const float2 st2 = a.stats[mc], cf = a.coef[mc];
            top = st2.x;
            scale = cf.x / st2.y;
            minus = cf.y;
            tok = a.tok[mc] - a.n_first - n0 - 32 * IT * wn - 4 * h;
          }
#pragma unroll
          for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[e] = (float)acc[i][j][4 * q + e];
                if constexpr (C::I8) {
                  v[e] *= sx * cs[i][q][e];
                  if (has_bias) v[e] += cb[i][q][e];
                }
                if constexpr (C::EPI == kTileCeGrad) {
                  if (has_bias) v[e] += cb[i][q][e];
                  // a logit of -inf: exp gives 0 for the others' maximum, and no 1[j = t] either
                  const float p = v[e] == -INFINITY ? 0.0f : exp_fast(v[e] - top) * scale;
                  const bool target = tok == 32 * i + 8 * q + e && v[e] != -INFINITY;
                  v[e] = p - (target ? minus : 0.0f);
                  at_target = target ? v[e] : at_target;
                }
              }
              *reinterpret_cast<uint2*>(to + 32 * (IT * wn + i) + 8 * q + 4 * h) =
                  make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            }
          if constexpr (C::EPI == kTileCeGrad) {
            if (m < M && tok >= 0 && tok < 32 * IT && (tok & 4) == 0)
              a.rest[m] = rest_bf16(at_target, bf16_lo(pack_bf16(at_target, 0.0f)));
          }
        }
      }
      __syncthreads();
      constexpr int kChunks = kW / 8, kRows = 32 * kJP * C::WM, kIters = kRows * kChunks / kTileThreads;
      const int c = tid % kChunks, n = n0 + 8 * c, width = C::EPI == kTileGated ? a.I : a.N;
      if (n >= width) continue;
      const bool whole = !C::I8 || ((a.N & 7) == 0 && n + 8 <= a.N);
#pragma unroll 8
      for (int it = 0; it < kIters; ++it) {
        const int row = tid / kChunks + it * (kTileThreads / kChunks);
        const int m = m0 + 32 * (JT * (row / (32 * kJP)) + j0) + row % (32 * kJP);
        if (m >= M) continue;
        const uint16_t* const from = stage + row * C::kOutPitch;
        uint16_t* const o = (uint16_t*)a.out + (int64_t)m * a.out_pitch + n;
        u32x4 w = *reinterpret_cast<const u32x4*>(from + (C::EPI == kTileGated ? 4 * kW : 0) + 8 * c);
        if constexpr (C::EPI == kTileCeGrad) {                   // columns past the vocabulary: zero operands
          if (n + 8 > a.N) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = n + 2 * e + 1 < a.N ? w[e] : n + 2 * e < a.N ? w[e] & 0xFFFFu : 0u;
          }
        }
        if (whole) {
          // logits and weight gradients are not read back here (32003 x 2080 of 333 tokens, whole step: 267 -> 254 us)
          if constexpr (C::I8 || QT) __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(o));
          else *reinterpret_cast<u32x4*>(o) = w;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < a.N) o[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
        if constexpr (C::EPI == kTileGated) {
          if (a.pair_rows != 0)
            *reinterpret_cast<u32x4*>(o + (int64_t)a.pair_rows * a.out_pitch) =
                *reinterpret_cast<const u32x4*>(from + 5 * kW + 8 * c);
          if (a.act != nullptr) *reinterpret_cast<u32x4*>(a.act + (int64_t)m * a.I + n) = w;
          if (a.h != nullptr) {
            float* const hp = a.h + (int64_t)m * 2 * a.I + n;
            const f32x4* const src = reinterpret_cast<const f32x4*>((const float*)from + 8 * c);
            *reinterpret_cast<f32x4*>(hp) = src[0];
            *reinterpret_cast<f32x4*>(hp + 4) = src[1];
            *reinterpret_cast<f32x4*>(hp + a.I) = src[kW / 4];
            *reinterpret_cast<f32x4*>(hp + a.I + 4) = src[kW / 4 + 1];
          }
        }
      }
    }
  }
}

// Tiles, as rows of m by columns of n (gated: half the columns of output) and workgroups a compute unit takes.
enum TileSize : int { kTile32, kTile64, kTile128, kTile192, kTile256 };
struct TileShape {
  int bm, bn, per_cu;
};
constexpr TileShape tile_shape(TileSize t) {
  return t == kTile32 ? TileShape{32, 128, 2} : t == kTile64 ? TileShape{64, 128, 2}
       : t == kTile128 ? TileShape{128, 128, 2} : t == kTile192 ? TileShape{192, 256, 1} : TileShape{256, 256, 1};
}
inline int64_t tile_count(TileSize t, int64_t M, int64_t N) {
  const TileShape s = tile_shape(t);
  return (M + s.bm - 1) / s.bm * ((N + s.bn - 1) / s.bn);
}

inline int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }   // a workspace's parts start at multiples of 256

constexpr int kTileCus = 256;      // fixed, so that a workspace's size does not depend on the device that is current

// The tile for an [M, N] product over `steps` steps, K split `splits` times.  Few rows: the least tile that holds
// them (bound by memory; two workgroups a compute unit keep more of it in flight).  Else by the time of a round of
// workgroups, as measured: 1.3 us a step and 8 us besides for 256 x 256, 1.0 and 7 for 192 x 256, 1.0 and 2.5
// for two of 128 x 128 (one's epilogue under the other's steps), or 0.65 and 6 where those have a compute
// unit each.  4096 x 28672 over 64 steps: 740 us in 256 x 256, 890 in 128 x 128; 333 x 32003 over 33: 59, 52 (192 x 256),
// 67; 333 x 11232 over 33: 46, 37, 32; 32003 x 2080 over 6: 76, 72, 67.
// 192 rows are not for a transposed m side (`whole`), whose rows of 192 columns do not fill a copy.
inline TileSize tile_size(int64_t M, int64_t N, int64_t steps, int64_t splits, bool whole = false) {
  if (M <= 32) return kTile32;
  if (M <= 64) return kTile64;
  const int64_t t256 = tile_count(kTile256, M, N) * splits, t128 = tile_count(kTile128, M, N) * splits;
  const double big = (double)((t256 + kTileCus - 1) / kTileCus) * (1.3 * (double)steps + 8.0);
  const double small = t128 <= kTileCus ? 0.65 * (double)steps + 6.0
                                        : (double)((t128 + 2 * kTileCus - 1) / (2 * kTileCus)) * (1.0 * (double)steps + 2.5);
  const int64_t t192 = tile_count(kTile192, M, N) * splits;
  const double mid = (double)((t192 + kTileCus - 1) / kTileCus) * (1.0 * (double)steps + 7.0);
  if (!whole && mid < big && mid < small) return kTile192;
  return small < big ? kTile128 : kTile256;
}

// Splits of K (in steps of 64) for an [M, N] product whose tiles do not fill the compute units: at least `least`
// steps each, the tile chosen with them.
struct TileSplit {
  TileSize size;
  int splits, k_split;
};
inline TileSplit tile_split(int64_t M, int64_t N, int64_t K, int64_t least, int64_t most) {
  const int64_t steps = (K + 63) / 64;
  TileSplit best = {tile_size(M, N, steps, 1), 1, 0};
  const TileShape shape = tile_shape(M > 64 ? kTile128 : best.size);
  const int64_t tiles = (M + shape.bm - 1) / shape.bm * ((N + shape.bn - 1) / shape.bn);
  int64_t s = kTileCus * shape.per_cu / tiles;
  s = s > most ? most : s;
  s = s > steps / least ? steps / least : s;
  if (s > 1) {
    const int64_t per = (steps + s - 1) / s;
    best.splits = (int)((steps + per - 1) / per);
    best.k_split = (int)per * 64;
    best.size = tile_size(M, N, per, best.splits);
  } else {
    best.k_split = (int)steps * 64;
  }
  return best;
}

// Floats that hold the parts of every [m, N] product, m <= M, that tile_split cuts in two or more (0: none is): a size
// that does not fall as M grows.  There are at most 2 kTileCus / tiles parts, and a tile is at most 128 x 128.
inline int64_t tile_split_floats(int64_t M, int64_t N, int64_t K, int64_t least, int64_t most) {
  int64_t s = (K + 63) / 64 / least;
  s = s > most ? most : s;
  const int64_t limit = (int64_t)kTileCus * 2 * 128 * 128;
  return s <= 1 ? 0 : s * M * N < limit ? s * M * N : limit;
}

// Eight columns from `at` of the sum of `splits` partial products `stride` floats apart, by 256 threads: thread
// t's wavefront adds every fourth part, the first wavefront the four sums.  Only lanes with `on` read; the sum
// is the first wavefront's.
__device__ __forceinline__ void tile_join(const float* __restrict__ parts, int64_t at, int64_t stride, int splits,
                                          bool on, float (&v)[8]) {
  __shared__ float sums[3][64][9];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  if (on) {
#pragma unroll 4
    for (int s = wave; s < splits; s += 4) {
      const f32x4* const p = reinterpret_cast<const f32x4*>(parts + s * stride + at);
      const f32x4 lo = p[0], hi = p[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] += lo[e];
        v[4 + e] += hi[e];
      }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[wave - 1][lane][e] = v[e];
  }
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += sums[w][lane][e];
  }
}

template <class C>
inline hipError_t launch_tile_cfg(TileArgs a, hipStream_t stream) {
  const int width = C::EPI == kTileGated ? C::BN / 2 : C::BN;
  const int n = C::EPI == kTileGated ? a.I : a.N;
  a.m_tiles = (a.M + C::BM - 1) / C::BM;
  a.n_tiles = (n + width - 1) / width;
  // While the m side fits an XCD's L2, tiles of n may be anywhere in K; a larger one is shared
  // through the L2 by workgroups of one XCD that are at the same step.
  a.turn_by_tile = (int64_t)a.M * a.K * (C::I8 ? 1 : 2) <= ((int64_t)2 << 20);
  const int64_t grid = (int64_t)a.m_tiles * a.n_tiles * a.splits;
  return launch_kernel((const void*)dense_tile_kernel<C>, dim3((unsigned)grid), dim3(kTileThreads), stream, a);
}

template <int EPI, bool PT, bool QT>
inline hipError_t launch_tile(const TileArgs& a, TileSize size, hipStream_t stream) {
  if constexpr (!QT) {
    if (size == kTile32) {
      // a wavefront of the gated kernel needs a tile of gates and one of ups
      if constexpr (EPI == kTileGated) return launch_tile_cfg<TileCfg<2, 1, 2, 2, PT, QT, EPI, 3>>(a, stream);
      else return launch_tile_cfg<TileCfg<1, 1, 4, 1, PT, QT, EPI, 4>>(a, stream);
    }
    if (size == kTile64) return launch_tile_cfg<TileCfg<2, 1, 2, 2, PT, QT, EPI, 3>>(a, stream);
  }
  if (size <= kTile128) return launch_tile_cfg<TileCfg<2, 2, 2, 2, PT, QT, EPI, 0>>(a, stream);
  if constexpr (!QT)
    if (size == kTile192) return launch_tile_cfg<TileCfg<4, 3, 2, 2, PT, QT, EPI, 0>>(a, stream);
  return launch_tile_cfg<TileCfg<4, 4, 2, 2, PT, QT, EPI, 0>>(a, stream);
}

}  // namespace nvfp4
