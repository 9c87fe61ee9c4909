// Streaming 16-row tiles of 4-bit weights through LDS, for the kernels whose
// wavefronts split K (gfx950).
//
// A wavefront owns the same NC chunks of 256 k of every row and keeps the
// activations of those k in registers; tiles of 16 rows pass by.  HBM streams at
// full rate only when each load instruction covers whole 128-byte lines of a
// row (eight lanes a row), which is not how the MFMA wants its operand (four
// lanes a row), so a tile's chunk (16 rows x 128 bytes) is copied straight to LDS by
// two such loads and read back in the operand layout, 16-byte pieces swizzled
// by the row so that the reads spread over the banks.  A ring of D tiles per
// wavefront is in flight; only the wavefront itself waits for it.
#pragma once

#include "nvfp4_device.hpp"

namespace nvfp4 {

constexpr int kSt4Chunk = 256;               // k per chunk
constexpr int kSt4Bytes = 2048;              // LDS bytes of a tile's chunk
typedef __attribute__((address_space(3))) void* st4_lds_t;

// s_waitcnt with vmcnt(n) alone, and lgkmcnt(0) alone (gfx9 encoding).
constexpr int st4_vm(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kSt4Lgkm0 = 0xC07F;

// Byte of a row from which lane l copies chunk c: piece (l % 8) ^ (l / 8).  Pieces past
// the row's end (K % 256 != 0) repeat its last one; their activations are zero.
template <typename Int>
__device__ __forceinline__ Int st4_offset(int c, Int pitch, int lane) {
  return min((Int)(kSt4Chunk / 2) * c + 16 * ((lane & 7) ^ (lane >> 3)), pitch - 16);
}

// Copy a tile's chunk into region, lane l from row l / 8 (at) and row 8 + l / 8 (below).
__device__ __forceinline__ void st4_copy_rows(const uint8_t* at, const uint8_t* below, uint8_t* region) {
  __builtin_amdgcn_global_load_lds((const void*)at, (st4_lds_t)region, 16, 0, 2 /* nontemporal */);
  __builtin_amdgcn_global_load_lds((const void*)below, (st4_lds_t)(region + 1024), 16, 0, 2 /* nontemporal */);
}

// The same for rows 0..15 of a tile (row index clamped to last).
__device__ __forceinline__ void st4_copy(const uint8_t* tile, int64_t pitch, int last, int c, uint8_t* region,
                                         int lane) {
  const uint8_t* const p = tile + st4_offset<int64_t>(c, pitch, lane);
  st4_copy_rows(p + min(lane >> 3, last) * pitch, p + min(8 + (lane >> 3), last) * pitch, region);
}

// Piece p (0..7) of the chunk for lane row r.
__device__ __forceinline__ u32x4 st4_read(const uint8_t* region, int r, int p) {
  return *reinterpret_cast<const u32x4*>(region + r * 128 + 16 * (p ^ (r & 7)));
}

// Barrier for LDS alone: loads in flight stay in flight.
__device__ __forceinline__ void st4_barrier() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(kSt4Lgkm0);
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}

}  // namespace nvfp4
