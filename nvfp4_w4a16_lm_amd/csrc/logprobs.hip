// Log probabilities of given tokens, with their rank, the entropy and the top
// alternatives, from the logits that the lm_head produced, and the gradient
// (gfx950).
//
// Forward.  For a row x[0..V) with temperature T, z = x / T, over the allowed
// tokens: lse = log sum_j exp(z_j), logprob = z_id - lse, H = -sum_j p_j log p_j.
// One pass over the row keeps, per lane, the running maximum m and the two sums
//   s = sum 2^(y_j),  t = sum 2^(y_j) y_j,   y_j = (x_j - m) log2(e) / T,
// rescaled when the maximum grows (s' = s a, t' = (t + s d) a with d = (m - m') log2(e) / T
// and a = 2^d); then lse = m / T + log s and H = log s - (t / s) ln 2.  The difference
// comes first: scaled logits rounded on their own would leave up to |z| 2^-24 between a
// logit and its own maximum, which no float32 power holds from |z| of 2^31 on (12
// operations a logit instead of 13, 2048 x 128256 at most 2 % faster, and NaN there).  Logits go to float32's largest, so half
// the difference is taken, and twice the scale: no finite pair overflows.
// The rank is a count of larger logits in the same pass.
//
// Top alternatives: each wavefront keeps its best 64 as one 64-bit key per
// lane, sorted, key = (order-preserving image of the logit, ~index), so equal
// logits order by the lower index and every comparison is exact.  A group of
// 16 logits per lane is only looked at when some lane's maximum reaches the
// bound so far; when many do, a bisection over the lanes' maxima raises the
// bound first (of 128 maxima about as many logits pass as are wanted).  What
// passes is appended to a buffer that is sorted when it fills (one insertion at
// a time into a sorted register list instead: 333 x 32003 with 64 alternatives
// 123 us).  Lists of two wavefronts or segments merge by a bitonic step:
// max(a[i], b[63 - i]), then six compare-exchanges.
//
// With few rows a row is split into segments, one workgroup each; a second
// kernel joins the segments' sums, counts and lists in segment order (no
// atomics, so results do not depend on timing).
//
// Many rows: 2048 x 128256 bf16 110 us (4.8 TB/s; the vector units are 80 % busy with
// 13 operations a logit, HBM close behind).  Few rows: launches and the
// lists; one row 13 us (9 us the segments, of which most is the first loads and the
// sort, 5 us the join), 64 x 151936 masked with 20 alternatives 25 us, 333 x 32003
// float32 with 64 alternatives 35 us (1.2 TB/s; most of it the lists).
//
// Backward.  d logprob / dz_j = 1[j = id] - p_j, dH / dz_j = -p_j (log p_j + H),
// dlse / dz_j = p_j: one read and one write per logit, p_j recomputed from lse.
//
// Rows start at any element (2-byte or 4-byte) alignment: the 16-byte accesses
// below are declared with the element's alignment.
#include <algorithm>

#include "nvfp4_device.hpp"
#include "nvfp4_launch.hpp"

namespace nvfp4 {

namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;
constexpr int kGroup16 = 16;                 // logits per lane and step
constexpr int kJoinWaves = 8;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLargest = 3.40282346638528859812e38f;
constexpr float kLeast = 1.40129846432481707092e-45f;    // 2^-149
constexpr float kLowest = -kLargest;         // a maximum of nothing: s = 0 tells it from a row of this value

constexpr int kBf16 = 0, kF16 = 1, kF32 = 2;

struct __attribute__((packed, aligned(2))) Vec16A2 { u32x4 v; };
struct __attribute__((packed, aligned(4))) Vec16A4 { u32x4 v; };

template <int DT> struct Elem;
template <> struct Elem<kBf16> {
  static constexpr int kBytes = 2, kPerVec = 8, kLowBits = 16;   // image bits below are alike
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  static __device__ __forceinline__ u32x4 load(const uint8_t* p) { return reinterpret_cast<const Vec16A2*>(p)->v; }
  static __device__ __forceinline__ void store(uint8_t* p, u32x4 v) { reinterpret_cast<Vec16A2*>(p)->v = v; }
  static __device__ __forceinline__ uint32_t bits(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b << 16); }
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(v[i]);
      f[2 * i + 1] = bf16_hi(v[i]);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
    return o;
  }
};
template <> struct Elem<kF16> {
  static constexpr int kBytes = 2, kPerVec = 8, kLowBits = 13;
  static constexpr uint32_t kNegInf = 0xFC00FC00u;
  static __device__ __forceinline__ u32x4 load(const uint8_t* p) { return reinterpret_cast<const Vec16A2*>(p)->v; }
  static __device__ __forceinline__ void store(uint8_t* p, u32x4 v) { reinterpret_cast<Vec16A2*>(p)->v = v; }
  static __device__ __forceinline__ uint32_t bits(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
  static __device__ __forceinline__ float value(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = v[i];                 // a value: bit_cast of a vector's element takes element 0
      const f16x2 h = __builtin_bit_cast(f16x2, w);
      f[2 * i] = (float)h[0];
      f[2 * i + 1] = (float)h[1];
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)f[2 * i], (_Float16)f[2 * i + 1]});
    return o;
  }
};
template <> struct Elem<kF32> {
  static constexpr int kBytes = 4, kPerVec = 4, kLowBits = 0;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  static __device__ __forceinline__ u32x4 load(const uint8_t* p) { return reinterpret_cast<const Vec16A4*>(p)->v; }
  static __device__ __forceinline__ void store(uint8_t* p, u32x4 v) { reinterpret_cast<Vec16A4*>(p)->v = v; }
  static __device__ __forceinline__ uint32_t bits(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b); }
  static __device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};

// Elements [j, V) of a row whose last vector is cut: the missing ones are -inf.
template <int DT>
__device__ __forceinline__ u32x4 load_tail(const uint8_t* row, int j, int V) {
  u32x4 v = {Elem<DT>::kNegInf, Elem<DT>::kNegInf, Elem<DT>::kNegInf, Elem<DT>::kNegInf};
#pragma unroll
  for (int e = 0; e < Elem<DT>::kPerVec; ++e) {
    if (j + e < V) {
      const uint32_t b = Elem<DT>::bits(row + (int64_t)(j + e) * Elem<DT>::kBytes);
      if (DT == kF32) {
        v[e & 3] = b;
      } else {
        const int w = (e >> 1) & 3;
        v[w] = (e & 1) ? ((v[w] & 0xFFFFu) | (b << 16)) : ((v[w] & 0xFFFF0000u) | b);
      }
    }
  }
  return v;
}

// A row's temperature as 1 / T; a temperature that is not greater than 0
// (greedy rows) counts as 1.
__device__ __forceinline__ float inv_temperature(const float* temps, int64_t row) {
  if (!temps) return 1.0f;
  const float t = temps[row];
  return t > 0.0f ? 1.0f / t : 1.0f;
}

// Twice log2(e) / T, from one division; a T so small that this overflows still
// leaves every other logit 2^-1000 behind.  At T = +inf it is float32's least value,
// not 0: finite differences come to 2^-20 at most, and -inf stays -inf.
__device__ __forceinline__ float base2_scale(const float* temps, int64_t row) {
  if (!temps) return 2.0f * kLog2e;
  const float t = temps[row];
  return t > 0.0f ? fmaxf(fminf(2.0f * kLog2e / t, kLargest), kLeast) : 2.0f * kLog2e;
}

// Half of x - m without overflow, given m / 2.
__device__ __forceinline__ float half_difference(float x, float half_m) { return __builtin_fmaf(x, 0.5f, -half_m); }

// ---------------------------------------------------------------------------
// Sorted lists of 64 keys, one per lane, best first; 0 = empty.
// ---------------------------------------------------------------------------
struct Key {
  uint32_t hi, lo;                           // order-preserving image of the logit; ~index
};

__device__ __forceinline__ bool key_gt(Key a, Key b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

__device__ __forceinline__ uint32_t key_image(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);          // -0 compares equal to +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t h) {
  return __uint_as_float((h >> 31) ? (h & 0x7FFFFFFFu) : ~h);
}

__device__ __forceinline__ Key key_xor(Key k, int d) {
  return Key{(uint32_t)__shfl_xor((int)k.hi, d, 64), (uint32_t)__shfl_xor((int)k.lo, d, 64)};
}

// 64 keys in any order, one per lane -> sorted, best first (bitonic).
__device__ __forceinline__ Key list_sort(Key k, int lane) {
#pragma unroll
  for (int size = 2; size <= 64; size <<= 1) {
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const Key o = key_xor(k, d);
      const bool keep_max = ((lane & d) == 0) == ((lane & size) == 0);
      if (key_gt(o, k) == keep_max) k = o;
    }
  }
  return k;
}

// Best 64 of two sorted lists, sorted.
__device__ __forceinline__ Key list_merge(Key a, Key b, int lane) {
  Key r;
  r.hi = (uint32_t)__shfl((int)b.hi, 63 - lane, 64);
  r.lo = (uint32_t)__shfl((int)b.lo, 63 - lane, 64);
  Key k = key_gt(a, r) ? a : r;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const Key o = key_xor(k, d);
    const bool keep_max = (lane & d) == 0;
    if (key_gt(o, k) == keep_max) k = o;
  }
  return k;
}

// A lower bound of the k-th best of the wavefront's logits: the largest T (its
// bits below `low` zero) that at least k of the 128 images a, b (two per lane,
// each the best of some of the lane's logits) reach; 0 if fewer than k are real.
__device__ __forceinline__ uint32_t kth_bound(uint32_t a, uint32_t b, int k, int low) {
  uint32_t t = 0;
  for (int bit = 31; bit >= low; --bit) {
    const uint32_t up = t | (1u << bit);
    if (__popcll(__ballot(a >= up)) + __popcll(__ballot(b >= up)) >= k) t = up;
  }
  return t;
}

// Candidates of a wavefront for its best k: at most 256 keys in LDS, in any
// order, and the value below which a logit need not be looked at.
struct Candidates {
  Key* keys;
  int count;
  float thr;

  // Keep the best k of them, sorted, and raise thr to the k-th.
  __device__ __forceinline__ Key compact(int k, int lane) {
    Key best = {0u, 0u};
    for (int c = 0; c < count; c += 64) {
      Key o = {0u, 0u};
      if (c + lane < count) o = keys[c + lane];
      o = list_sort(o, lane);
      best = c == 0 ? o : list_merge(best, o, lane);
    }
    const uint32_t kth = (uint32_t)__builtin_amdgcn_readlane((int)best.hi, k - 1);
    count = min(count, k);
    if (lane < k) keys[lane] = best;                     // the wavefront's own LDS: in order
    if (kth != 0) thr = fmaxf(thr, key_value(kth));
    return lane < k ? best : Key{0u, 0u};
  }
};

// Softmax sums of a set of logits.
struct Sums {
  float raw, s, t;                           // largest logit, sum 2^y, sum 2^y y
};

// Beyond 2^-1000 the factor is 0 in float32; bounded there, since an infinite
// distance, or one that overflows times s, would make t NaN.  A NaN stays in s.
__device__ __forceinline__ void rescale(Sums& q, float to, float c2) {
  const float d = fmaxf(half_difference(q.raw, 0.5f * to) * c2, -1000.0f);  // <= 0
  const float a = __builtin_amdgcn_exp2f(d);
  q.t = __builtin_fmaf(q.s, d, q.t) * a;
  q.s *= a;
  q.raw = to;
}

__device__ __forceinline__ Sums combine(Sums a, Sums b, float c2) {
  const float to = fmaxf(a.raw, b.raw);
  rescale(a, to, c2);
  rescale(b, to, c2);
  return Sums{to, a.s + b.s, a.t + b.t};
}

__device__ __forceinline__ Sums wave_combine(Sums a, float c2) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    Sums b;
    b.raw = __shfl_xor(a.raw, d, 64);
    b.s = __shfl_xor(a.s, d, 64);
    b.t = __shfl_xor(a.t, d, 64);
    a = combine(a, b, c2);
  }
  return a;
}

}  // namespace

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------
namespace {

// The given token's logit of a row: NaN-free flag `given` tells whether there
// is one; a token that is not allowed counts as -inf.
template <int DT>
__device__ __forceinline__ float token_logit(const LogprobsArgs& a, const uint8_t* row, int64_t i, bool* given) {
  *given = false;
  if (!a.tok) return 0.0f;
  const int id = a.tok[i];
  if (id < 0 || id >= a.V) return 0.0f;
  *given = true;
  const float x = Elem<DT>::value(Elem<DT>::bits(row + (int64_t)id * Elem<DT>::kBytes));
  if (a.allowed && !((a.allowed[i * a.mask_words + (id >> 5)] >> (id & 31)) & 1u)) return -INFINITY;
  return x;
}

// The row's outputs from its sums, count and list (one wavefront); xt = the
// given token's logit, if there is one.
__device__ __forceinline__ void finish_row(const LogprobsArgs& a, int64_t i, Sums q, int larger, Key k, bool given,
                                           float xt, float invt, int lane) {
  const bool empty = q.s == 0.0f;            // nothing allowed or finite, and no NaN: a maximum adds 1
  const float logs = logf(q.s);
  auto lp_of = [&](float x) {
    if (empty) return -INFINITY;
    const float z = x == -INFINITY ? x : 2.0f * (half_difference(x, 0.5f * q.raw) * invt);
    return z - logs;
  };
  if (lane == 0) {
    if (a.token_logprob) a.token_logprob[i] = given ? lp_of(xt) : 0.0f;
    if (a.token_rank) a.token_rank[i] = given ? larger + 1 : 0;
    if (a.lse) a.lse[i] = empty ? -INFINITY : __builtin_fmaf(q.raw, invt, logs);
    if (a.entropy) a.entropy[i] = empty ? 0.0f : logs - q.t / q.s * kLn2;
  }
  if (lane < a.topk) {
    const bool some = k.hi != 0;
    a.top_ids[i * a.topk + lane] = some ? (int32_t)~k.lo : -1;
    a.top_logprobs[i * a.topk + lane] = some ? lp_of(key_value(k.hi)) : -INFINITY;
  }
}

}  // namespace

template <int DT, bool MASK>
__global__ __launch_bounds__(kLpThreads) void logprobs_kernel(LogprobsArgs a) {
  using E = Elem<DT>;
  constexpr int VE = E::kPerVec, U = kGroup16 / VE;
  __shared__ Sums sh_sums[kLpWaves];
  __shared__ int sh_larger[kLpWaves];
  __shared__ Key sh_keys[kLpWaves][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t i = blockIdx.x / a.segs;
  const int seg = (int)(blockIdx.x - i * a.segs);
  const uint8_t* const row = a.x + i * a.row_stride * E::kBytes;
  const uint32_t* const bits = MASK ? a.allowed + i * a.mask_words : nullptr;
  const int V = a.V;
  const int nv = (V + VE - 1) / VE, full = V / VE;       // vectors, whole vectors
  const int v0 = seg * a.seg_vecs, v1 = min(nv, v0 + a.seg_vecs);
  bool given;
  const float xt_lane = token_logit<DT>(a, row, i, &given);
  const float xt = given ? xt_lane : INFINITY;           // without a token nothing is larger
  const float c2 = base2_scale(a.temps, i);

  Sums q = {kLowest, 0.0f, 0.0f};
  float half = 0.5f * kLowest;
  int larger = 0;
  const int kk = a.topk;
  Candidates cand = {sh_keys[wave], 0, kLowest};         // -inf and NaN never pass

  auto load = [&](int v) -> u32x4 {
    if (v < min(v1, full)) return E::load(row + (int64_t)v * 16);
    if (v < v1) return load_tail<DT>(row, v * VE, V);
    return u32x4{E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf};
  };

  u32x4 cur[U], next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) cur[u] = load(v0 + kLpThreads * u + tid);
  for (int vb = v0; vb < v1; vb += kLpThreads * U) {
    const bool more = vb + kLpThreads * U < v1;
    if (more) {
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = load(vb + kLpThreads * (U + u) + tid);
    }
    float f[kGroup16];
#pragma unroll
    for (int u = 0; u < U; ++u) E::unpack(cur[u], f + VE * u);
    if (MASK) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j0 = (vb + kLpThreads * u + tid) * VE;
        const uint32_t w = j0 < V ? bits[j0 >> 5] >> (j0 & 31) : 0u;
#pragma unroll
        for (int e = 0; e < VE; ++e) f[VE * u + e] = ((w >> e) & 1u) ? f[VE * u + e] : -INFINITY;
      }
    }
    float ga = f[0], gb = f[kGroup16 / 2];
#pragma unroll
    for (int e = 1; e < kGroup16 / 2; ++e) {
      ga = fmaxf(ga, f[e]);
      gb = fmaxf(gb, f[kGroup16 / 2 + e]);
    }
    const float g = fmaxf(ga, gb);
    if (g > q.raw) {
      rescale(q, g, c2);
      half = 0.5f * g;
    }
#pragma unroll
    for (int e = 0; e < kGroup16; ++e) {
      const float y = half_difference(f[e], half) * c2;
      const float p = __builtin_amdgcn_exp2f(y);
      q.s += p;
      q.t = __builtin_fmaf(p, fmaxf(y, -1000.0f), q.t);  // 2^y is 0 there; a NaN stays in s
      larger += __popcll(__ballot(f[e] > xt));
    }
    if (kk > 0 && __ballot(g >= cand.thr) != 0) {
      const float before = cand.thr;
      if (__popcll(__ballot(ga >= before)) + __popcll(__ballot(gb >= before)) > kk) {
        const uint32_t t = kth_bound(ga > -INFINITY ? key_image(ga) : 0u, gb > -INFINITY ? key_image(gb) : 0u, kk,
                                     E::kLowBits);
        if (t > key_image(before)) cand.thr = key_value(t);
      }
#pragma unroll
      for (int e = 0; e < kGroup16; ++e) {
        const uint64_t pass = __ballot(f[e] >= cand.thr);
        if (pass != 0) {
          if (f[e] >= cand.thr) {
            const int j = (vb + kLpThreads * (e / VE) + tid) * VE + e % VE;
            const int at = cand.count + __popcll(pass & (((uint64_t)1 << lane) - 1));
            cand.keys[at] = Key{key_image(f[e]), ~(uint32_t)j};
          }
          cand.count += __popcll(pass);
          if (cand.count > 192) cand.compact(kk, lane);   // the next 64 fit
        }
      }
      // later groups have higher indices: of equal logits the k here stay ahead
      if (cand.thr > before) cand.thr = key_value(key_image(cand.thr) + 1);
    }
    if (more) {
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = next[u];
    }
  }

  // wavefronts -> workgroup
  q = wave_combine(q, c2);
  if (lane == 0) {
    sh_sums[wave] = q;
    sh_larger[wave] = larger;
  }
  Key key = {0u, 0u};
  if (kk > 0) {
    key = cand.compact(kk, lane);
    sh_keys[wave][lane] = key;
  }
  __syncthreads();
  if (wave != 0) return;
  Sums total = sh_sums[0];
  int count = sh_larger[0];
#pragma unroll
  for (int w = 1; w < kLpWaves; ++w) {
    total = combine(total, sh_sums[w], c2);
    count += sh_larger[w];
  }
  if (kk > 0) {
#pragma unroll
    for (int w = 1; w < kLpWaves; ++w) key = list_merge(key, sh_keys[w][lane], lane);
  }
  if (a.segs == 1) {
    finish_row(a, i, total, count, key, given, xt_lane, inv_temperature(a.temps, i), lane);
    return;
  }
  LogprobsPart* const part = a.parts + blockIdx.x;
  if (lane == 0) *part = LogprobsPart{total.raw, total.s, total.t, count};
  if (lane < kk) reinterpret_cast<Key*>(a.part_keys)[(int64_t)blockIdx.x * kk + lane] = key;
}

// Joins a row's segments: lane q of wavefront 0 takes segments q, q + 64, ...
// in order; wavefront w merges the lists of segments w, w + 8, ...
template <int DT>
__global__ __launch_bounds__(64 * kJoinWaves) void logprobs_join_kernel(LogprobsArgs a) {
  __shared__ Key sh_keys[kJoinWaves][64];
  __shared__ Sums sh_sums;
  __shared__ int sh_larger;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t i = blockIdx.x;
  const int kk = a.topk;
  bool given;                                            // looked up now, used at the end
  const float xt = token_logit<DT>(a, a.x + i * a.row_stride * Elem<DT>::kBytes, i, &given);
  const float invt = inv_temperature(a.temps, i), c2 = base2_scale(a.temps, i);
  // the last wavefront adds the sums while the others merge lists, or the first where there are none
  const bool adds = wave == (kk > 0 ? kJoinWaves - 1 : 0);
  LogprobsPart first = {kLowest, 0.0f, 0.0f, 0};
  if (adds && lane < a.segs) first = a.parts[i * a.segs + lane];
  Sums q;
  int count;
  auto add_parts = [&]() {
    q = Sums{first.raw, first.s, first.t};
    count = first.larger;
    for (int g = lane + 64; g < a.segs; g += 64) {
      const LogprobsPart p = a.parts[i * a.segs + g];
      q = combine(q, Sums{p.raw, p.s, p.t}, c2);
      count += p.larger;
    }
    q = wave_combine(q, c2);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) count += __shfl_xor(count, d, 64);
  };
  Key key = {0u, 0u};
  if (kk > 0) {
    const Key* const lists = reinterpret_cast<const Key*>(a.part_keys) + i * a.segs * kk;
    for (int g = wave; g < a.segs; g += kJoinWaves) {
      Key o = {0u, 0u};
      if (lane < kk) o = lists[(int64_t)g * kk + lane];
      key = g == wave ? o : list_merge(key, o, lane);
    }
    sh_keys[wave][lane] = key;
#pragma unroll
    for (int half = kJoinWaves / 2; half > 0; half >>= 1) {
      __syncthreads();
      if (wave < half) {
        key = list_merge(key, sh_keys[wave + half][lane], lane);
        sh_keys[wave][lane] = key;
      } else if (half == kJoinWaves / 2 && adds) {
        add_parts();
        if (lane == 0) {
          sh_sums = q;
          sh_larger = count;
        }
      }
    }
    q = sh_sums;
    count = sh_larger;
  } else if (adds) {
    add_parts();
  }
  if (wave != 0) return;
  finish_row(a, i, q, count, key, given, xt, invt, lane);
}

// ---------------------------------------------------------------------------
// Backward: dx_j = (1 / T) [ g_lp 1[j = id] + p_j (g_lse - g_lp - g_H (log p_j + H)) ],
// log p_j = x_j / T - lse; 0 where the token is not allowed or its logit is
// -inf.  A workgroup owns a run of one row's vectors.  HBM bounds it: 1024 x 128256
// bf16 95 us (5.5 TB/s read and written).
//
// lse is a float32, so p_j is off by half its last place: 2^-15 of p_j below |lse| = 1024,
// 2^-12 below 8192, and nothing is right once |lse| passes 2^24 (low temperatures, large
// logits).  From 1024 on (8192 for bf16, whose own rounding is 2^-9) one of a row's
// workgroups takes the whole row and sums it again relative to its maximum, as the
// forward does, before it writes; the others leave.  Which one goes by the row, or
// with a multiple of eight segments all of them would land on one XCD.
// Such rows alone, 128256 bf16: 1 row 45 us (7 ordinary), 1024 rows 202 us (97).
// ---------------------------------------------------------------------------
namespace {

// A row's sums by one workgroup.
template <int DT, bool MASK>
__device__ Sums row_sums(const uint8_t* row, const uint32_t* bits, int V, float c2, Sums* sh) {
  using E = Elem<DT>;
  constexpr int VE = E::kPerVec, U = 4;
  const int tid = threadIdx.x, nv = (V + VE - 1) / VE, full = V / VE;
  auto load = [&](int v) -> u32x4 {
    if (v < full) return E::load(row + (int64_t)v * 16);
    if (v < nv) return load_tail<DT>(row, v * VE, V);
    return u32x4{E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf};
  };
  Sums q = {kLowest, 0.0f, 0.0f};
  u32x4 cur[U], next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) cur[u] = load(kLpThreads * u + tid);
  for (int vb = 0; vb < nv; vb += kLpThreads * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) next[u] = load(vb + kLpThreads * (U + u) + tid);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j0 = (vb + kLpThreads * u + tid) * VE;
      const uint32_t w = MASK && j0 < V ? bits[j0 >> 5] >> (j0 & 31) : 0xFFFFFFFFu;
      float f[VE];
      E::unpack(cur[u], f);
      float g = kLowest;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        if (MASK && !((w >> e) & 1u)) f[e] = -INFINITY;
        g = fmaxf(g, f[e]);
      }
      if (g > q.raw) rescale(q, g, c2);
      const float half = 0.5f * q.raw;
#pragma unroll
      for (int e = 0; e < VE; ++e) q.s += __builtin_amdgcn_exp2f(half_difference(f[e], half) * c2);
      cur[u] = next[u];
    }
  }
  q = wave_combine(q, c2);
  if ((tid & 63) == 0) sh[tid >> 6] = q;
  __syncthreads();
  q = sh[0];
#pragma unroll
  for (int w = 1; w < kLpWaves; ++w) q = combine(q, sh[w], c2);
  return q;
}

}  // namespace

template <int DT, bool MASK>
__global__ __launch_bounds__(kLpThreads) void logprobs_backward_kernel(LogprobsBackwardArgs a) {
  using E = Elem<DT>;
  constexpr int VE = E::kPerVec, U = kGroup16 / VE;
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / a.segs;
  const int seg = (int)(blockIdx.x - i * a.segs);
  const uint8_t* const row = a.x + i * a.row_stride * E::kBytes;
  uint8_t* const out = a.dx + i * a.dx_stride * E::kBytes;
  const uint32_t* const bits = MASK ? a.allowed + i * a.mask_words : nullptr;
  const int V = a.V;
  const int nv = (V + VE - 1) / VE, full = V / VE;
  int v0 = seg * a.seg_vecs, v1 = min(nv, v0 + a.seg_vecs);
  const float invt = inv_temperature(a.temps, i);
  // what 1 / T lost in rounding, so that x / T - lse is right to its own size
  // (log p of a likely token is a small difference of the two)
  float invt_lo = a.temps && a.temps[i] > 0.0f ? __builtin_fmaf(-a.temps[i], invt, 1.0f) * invt : 0.0f;
  if (!(fabsf(invt_lo) < INFINITY)) invt_lo = 0.0f;
  const float lse = a.lse[i];
  const bool empty = lse == -INFINITY;
  float top = 0.0f, base = lse;                          // log p = (x - top) / T - base
  __shared__ Sums sh_sums[kLpWaves];
  if (fabsf(lse) >= (DT == kBf16 ? 8192.0f : 1024.0f) && !empty) {   // the same for every workgroup of the row
    if (seg != (int)(i % a.segs)) return;
    v0 = 0;
    v1 = nv;
    const Sums q = row_sums<DT, MASK>(row, bits, V, base2_scale(a.temps, i), sh_sums);
    top = q.raw;
    base = logf(q.s);
  }
  const int id = a.tok ? a.tok[i] : -1;
  const bool given = id >= 0 && id < V;
  const float glp = given && a.dlogprob ? a.dlogprob[i] : 0.0f;
  const float gent = a.dentropy ? a.dentropy[i] : 0.0f;
  const float glse = a.dlse ? a.dlse[i] : 0.0f;
  const float b0 = glse - glp - (a.dentropy ? gent * a.entropy[i] : 0.0f);

  auto load = [&](int v) -> u32x4 {
    if (v < min(v1, full)) return E::load(row + (int64_t)v * 16);
    if (v < v1) return load_tail<DT>(row, v * VE, V);
    return u32x4{E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf};
  };
  u32x4 cur[U], next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) cur[u] = load(v0 + kLpThreads * u + tid);
  for (int vb = v0; vb < v1; vb += kLpThreads * U) {
    const bool more = vb + kLpThreads * U < v1;
    if (more) {
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = load(vb + kLpThreads * (U + u) + tid);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = vb + kLpThreads * u + tid, j0 = v * VE;
      if (v < v1) {
        float f[VE], d[VE];
        E::unpack(cur[u], f);
        const uint32_t w = MASK ? bits[j0 >> 5] >> (j0 & 31) : 0xFFFFFFFFu;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          if (MASK && !((w >> e) & 1u)) f[e] = -INFINITY;
          const float x = f[e] - top;
          const float lp = __builtin_fmaf(x, invt_lo, __builtin_fmaf(x, invt, -base));
          const float p = __builtin_amdgcn_exp2f(lp * kLog2e);
          d[e] = p * __builtin_fmaf(fmaxf(lp, -1000.0f), -gent, b0);
          if (f[e] == -INFINITY || empty) d[e] = 0.0f;
        }
        if (given && id >= j0 && id < j0 + VE && !empty) {
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (id == j0 + e && f[e] != -INFINITY) d[e] += glp;
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) d[e] *= invt;       // last: the factors times 1 / T could overflow beside p = 0
        const u32x4 o = E::pack(d);
        if (v < full) {
          E::store(out + (int64_t)v * 16, o);
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            if (j0 + e < V) {
              uint8_t* const q = out + (int64_t)(j0 + e) * E::kBytes;
              if (DT == kF32)
                *reinterpret_cast<uint32_t*>(q) = o[e & 3];
              else
                *reinterpret_cast<uint16_t*>(q) = (uint16_t)(o[(e >> 1) & 3] >> (16 * (e & 1)));
            }
          }
        }
      }
    }
    if (more) {
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = next[u];
    }
  }
}

// ---------------------------------------------------------------------------
// Launchers.
// ---------------------------------------------------------------------------
namespace {

int elem_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }

}  // namespace

// Segments per row: 2048 workgroups fill the GPU (eight on each of 256 compute
// units); with fewer rows a row is cut, in pieces of at least one step of a
// workgroup (16 logits per thread).  64 x 151936 masked, 20 alternatives: aiming
// at 512 / 1024 / 2048 / 4096 workgroups 29.8 / 28.3 / 25.9 / 30.1 us.
int64_t logprobs_segments(int64_t M, int64_t V) {
  const int64_t rows = std::max<int64_t>(M, 1);
  const int64_t steps = (V + kLpThreads * kGroup16 - 1) / (kLpThreads * kGroup16);
  const int64_t want = (2048 + rows - 1) / rows;
  const int64_t per = std::max<int64_t>(1, (steps + want - 1) / want);   // steps per segment
  return (steps + per - 1) / per;
}

int64_t logprobs_workspace_bytes(int64_t M, int64_t V, int64_t topk) {
  const int64_t segs = logprobs_segments(M, V);
  if (segs == 1) return 16;
  return std::max<int64_t>(16, M * segs * ((int64_t)sizeof(LogprobsPart) + 8 * topk));   // 0 would be a refusal
}

hipError_t launch_logprobs(LogprobsArgs a, int dtype, int64_t M, void* workspace, hipStream_t stream) {
  const int ve = 16 / elem_bytes(dtype);
  const int64_t nv = ((int64_t)a.V + ve - 1) / ve;
  const int64_t step = (int64_t)kLpThreads * kGroup16 / ve;            // vectors per step
  const int64_t steps = (nv + step - 1) / step;
  a.segs = (int)logprobs_segments(M, a.V);
  a.seg_vecs = (int)(step * ((steps + a.segs - 1) / a.segs));
  a.parts = static_cast<LogprobsPart*>(workspace);
  a.part_keys = a.parts ? reinterpret_cast<uint64_t*>(a.parts + M * a.segs) : nullptr;
  const bool mask = a.allowed != nullptr;
  const void* fn = nullptr;
  switch (dtype) {
    case kBf16: fn = mask ? (const void*)logprobs_kernel<kBf16, true> : (const void*)logprobs_kernel<kBf16, false>; break;
    case kF16: fn = mask ? (const void*)logprobs_kernel<kF16, true> : (const void*)logprobs_kernel<kF16, false>; break;
    default: fn = mask ? (const void*)logprobs_kernel<kF32, true> : (const void*)logprobs_kernel<kF32, false>; break;
  }
  hipError_t e = launch_kernel(fn, dim3((unsigned)(M * a.segs)), dim3(kLpThreads), stream, a);
  if (e != hipSuccess || a.segs == 1) return e;
  fn = dtype == kBf16 ? (const void*)logprobs_join_kernel<kBf16>
       : dtype == kF16 ? (const void*)logprobs_join_kernel<kF16>
                       : (const void*)logprobs_join_kernel<kF32>;
  return launch_kernel(fn, dim3((unsigned)M), dim3(64 * kJoinWaves), stream, a);
}

hipError_t launch_logprobs_backward(LogprobsBackwardArgs a, int dtype, int64_t M, hipStream_t stream) {
  const int ve = 16 / elem_bytes(dtype);
  const int64_t nv = ((int64_t)a.V + ve - 1) / ve;
  const int64_t step = (int64_t)kLpThreads * kGroup16 / ve;
  const int64_t steps = (nv + step - 1) / step;
  // two steps per workgroup, so that the second one's loads overlap the first
  // (more only where the grid would pass 2^23 workgroups)
  int64_t per = steps > 1 ? 2 : 1;
  while (per < steps && M * ((steps + per - 1) / per) > ((int64_t)1 << 23)) per *= 2;
  a.seg_vecs = (int)(step * per);
  a.segs = (int)((steps + per - 1) / per);
  const bool mask = a.allowed != nullptr;
  const void* fn = nullptr;
  switch (dtype) {
    case kBf16:
      fn = mask ? (const void*)logprobs_backward_kernel<kBf16, true> : (const void*)logprobs_backward_kernel<kBf16, false>;
      break;
    case kF16:
      fn = mask ? (const void*)logprobs_backward_kernel<kF16, true> : (const void*)logprobs_backward_kernel<kF16, false>;
      break;
    default:
      fn = mask ? (const void*)logprobs_backward_kernel<kF32, true> : (const void*)logprobs_backward_kernel<kF32, false>;
      break;
  }
  return launch_kernel(fn, dim3((unsigned)(M * a.segs)), dim3(kLpThreads), stream, a);
}

}  // namespace nvfp4
