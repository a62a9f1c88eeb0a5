// What the kernels over 4-bit weights with group scales share: units of 32 columns (16
// bytes of codes), steps of 16 units, and the lane layout of the 4x4x4 matrix product.
#pragma once

#include "common.h"

namespace lvq {

constexpr int kStepUnits = 16; // units of 32 columns per step

// log2 of the units of 32 columns that share a scale; 31 for one scale per row
inline int group_shift(int group) {
  return group == 0 ? 31 : group == 32 ? 0 : group == 64 ? 1 : group == 128 ? 2
       : group == 256 ? 3 : -1;
}
inline int group_count(int cols, int group) { return group ? (cols + group - 1) / group : 1; }

inline int units_of(int cols) { return (cols + 31) / 32; }
inline int steps_of(int cols) { return (units_of(cols) + 15) / 16; }
__host__ __device__ inline int groups_of(int units, int shift) {  // units > 0
  return ((units - 1) >> shift) + 1;
}

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef int int4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float float2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float f16_to_f32(uint32_t b) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t q4_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

// The pairs (x0, x4) (x2, x6) (x1, x5) (x3, x7) of eight fp16.
__device__ __forceinline__ u32x4_t pair_order(u32x4_t d) {
  return u32x4_t{__builtin_amdgcn_perm(d.z, d.x, 0x05040100u),
                 __builtin_amdgcn_perm(d.w, d.y, 0x05040100u),
                 __builtin_amdgcn_perm(d.z, d.x, 0x07060302u),
                 __builtin_amdgcn_perm(d.w, d.y, 0x07060302u)};
}

// v plus its counterparts in the other 15 blocks of four lanes: rotations inside
// a row of 16 lanes, then rows swapped pairwise.  Each step adds the same two
// values on both sides (blocks two apart first, then the two pair sums), so
// every lane ends with the same bits.
__device__ __forceinline__ float sum_blocks(float v) {
  v = dpp_add<0x128, 0xF>(v);  // row_ror:8
  v = dpp_add<0x124, 0xF>(v);  // row_ror:4
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
  u = __builtin_bit_cast(uint32_t, v);
  auto q = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)q[0]) + __builtin_bit_cast(float, (uint32_t)q[1]);
}

}  // namespace lvq
