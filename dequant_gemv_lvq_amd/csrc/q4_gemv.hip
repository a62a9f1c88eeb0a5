// 4-bit matvec with group scales (q4_gemv, q4_gemv_q8).
//
//   y[b][r] = sum_g s_rg (sum_(c in g) q_rc x_bc - z_rg sum_(c in g) x_bc)
//
// One wave per row; a lane takes units of 32 columns (16 bytes of codes), 64
// units apart, multiplies in fp32 and applies the unit's scale to the unit's
// sum.  The first, plain form of the kernel.

#include "common.h"

namespace lvq {

int zero_output(float* y, size_t n, hipStream_t st);

enum Q4X { kQ4F16 = 0, kQ4I8 = 1, kQ4E4M3 = 2 };

// log2 of the units of 32 columns that share a scale; 31 for one scale per row
inline int group_shift(int group) {
  return group == 0 ? 31 : group == 32 ? 0 : group == 64 ? 1 : group == 128 ? 2
       : group == 256 ? 3 : -1;
}
inline int group_count(int cols, int group) { return group ? (cols + group - 1) / group : 1; }

struct Q4Args {
  const uint8_t* codes;
  const uint16_t* scale;
  const uint16_t* zero;
  int gshift, groups, rows, cols, nunits;
  const void* x;
  const float* xscale;
  int xshift, xgroups;
  float* y;
};

__device__ __forceinline__ float f16_to_f32(uint16_t b) {
  return (float)__builtin_bit_cast(_Float16, b);
}

template <int B, int X>
__global__ void __launch_bounds__(256) q4_gemv_kernel(Q4Args a) {
  const int lane = threadIdx.x & (kWave - 1);
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.rows) return;
  float acc[B];
  for (int bb = 0; bb < B; ++bb) acc[bb] = 0.f;
  for (int u = lane; u < a.nunits; u += kWave) {
    const uint4 w = ((const uint4*)a.codes)[(size_t)row * a.nunits + u];
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    const size_t g = (size_t)row * a.groups + (u >> a.gshift);
    const float s = f16_to_f32(a.scale[g]);
    const float z = a.zero ? f16_to_f32(a.zero[g]) : 8.f;
    float t[B];
    for (int bb = 0; bb < B; ++bb) t[bb] = 0.f;
    for (int n = 0; n < 32; ++n) {
      const int c = u * 32 + n;
      if (c >= a.cols) break;
      const float q = (float)((ww[n >> 3] >> (4 * (n & 7))) & 15u) - z;
      for (int bb = 0; bb < B; ++bb) {
        const size_t i = (size_t)bb * a.cols + c;
        float xv;
        if (X == kQ4F16) xv = f16_to_f32(((const uint16_t*)a.x)[i]);
        else if (X == kQ4I8) xv = (float)((const int8_t*)a.x)[i];
        else xv = __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)a.x)[i], 0);
        t[bb] += q * xv;
      }
    }
    for (int bb = 0; bb < B; ++bb) {
      float sx = s;
      if (X != kQ4F16) sx *= a.xscale[(size_t)bb * a.xgroups + (u >> a.xshift)];
      acc[bb] += sx * t[bb];
    }
  }
  for (int bb = 0; bb < B; ++bb) {
    const float tot = wave_sum_lane63(acc[bb]);
    if (lane == kWave - 1) a.y[(size_t)bb * a.rows + row] = tot;
  }
}

template <int X>
int launch_q4(const Q4Args& a, int batch, hipStream_t st) {
  const dim3 grid((unsigned)((a.rows + 3) / 4)), block(256);
  clear_hip_error();
  switch (batch) {
    case 1: hipLaunchKernelGGL((q4_gemv_kernel<1, X>), grid, block, 0, st, a); break;
    case 2: hipLaunchKernelGGL((q4_gemv_kernel<2, X>), grid, block, 0, st, a); break;
    case 3: hipLaunchKernelGGL((q4_gemv_kernel<3, X>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((q4_gemv_kernel<4, X>), grid, block, 0, st, a); break;
  }
  return launch_status();
}

// The checks both entry points make, and the launch.
int q4_run(const uint8_t* codes, const uint16_t* scale, const uint16_t* zero, int group, int rows,
           int cols, const void* x, int xkind, const float* x_scale, int x_group, float* y,
           int batch, hipStream_t st) {
  if (rows < 0 || cols < 0) return LVQ_E_SHAPE;
  const int gs = group_shift(group), xs = group_shift(x_group);
  if (gs < 0 || xs < 0) return LVQ_E_SHAPE;
  const int e = check_batch(batch);
  if (e) return e;
  if (!y || (rows && cols && (!codes || !scale || !x || (xkind != kQ4F16 && !x_scale))))
    return LVQ_E_NULL;
  if (!aligned16(codes) || !aligned16(scale) || !aligned16(zero) || !aligned16(x) ||
      !aligned16(x_scale) || !aligned16(y))
    return LVQ_E_ALIGN;
  if ((long long)batch * cols > 65536) return LVQ_E_SHAPE;
  if (rows == 0) return LVQ_OK;
  const size_t ybytes = (size_t)batch * rows * 4;
  if (ranges_overlap(y, ybytes, x, (size_t)batch * cols * (xkind == kQ4F16 ? 2 : 1)) ||
      ranges_overlap(y, ybytes, x_scale, (size_t)batch * group_count(cols, x_group) * 4))
    return LVQ_E_SHAPE;
  if (cols == 0) return zero_output(y, (size_t)batch * rows, st);
  Q4Args a;
  a.codes = codes, a.scale = scale, a.zero = zero;
  a.gshift = gs, a.groups = group_count(cols, group);
  a.rows = rows, a.cols = cols, a.nunits = (cols + 31) / 32;
  a.x = x, a.xscale = x_scale;
  a.xshift = xs, a.xgroups = group_count(cols, x_group);
  a.y = y;
  if (xkind == kQ4F16) return launch_q4<kQ4F16>(a, batch, st);
  if (xkind == kQ4I8) return launch_q4<kQ4I8>(a, batch, st);
  return launch_q4<kQ4E4M3>(a, batch, st);
}

}  // namespace lvq

using namespace lvq;

extern "C" int q4_gemv(const uint8_t* codes, const uint16_t* scale, const uint16_t* zero,
                       int group, int rows, int cols, const uint16_t* x, float* y, int batch,
                       void* stream) {
  return q4_run(codes, scale, zero, group, rows, cols, x, kQ4F16, nullptr, 0, y, batch,
                (hipStream_t)stream);
}

extern "C" int q4_gemv_q8(const uint8_t* codes, const uint16_t* scale, const uint16_t* zero,
                          int group, int rows, int cols, const void* x, int x_type,
                          const float* x_scale, int x_group, float* y, int batch, void* stream) {
  if (x_type != LVQ_I8 && x_type != LVQ_E4M3) return LVQ_E_SHAPE;
  return q4_run(codes, scale, zero, group, rows, cols, x, x_type == LVQ_I8 ? kQ4I8 : kQ4E4M3,
                x_scale, x_group, y, batch, (hipStream_t)stream);
}
