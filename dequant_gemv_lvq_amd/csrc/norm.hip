// The transforms between two projections of a decoder block: the
// root-mean-square norm of a residual stream (lvq_rms_norm) and the gated
// activation (lvq_silu_mul), with fp16 or 8-bit outputs.
//
//   rms_norm   h = x + residual, out = h (mean h^2 + eps)^-1/2 w
//   silu_mul   out = g / (1 + e^-g) u
//   8 bits     a = max |out| over a group, scale = a / M, code = rne(out M / a)
//
// Both are streams: a few operations per value, so the bytes and, for the few
// rows of a decode step, the launch and one round of memory latency bound
// them.  A thread owns chunks of 8 consecutive columns (16 bytes of fp16, 32 of
// fp32): every array is read once into registers, the statistics are taken
// there, and every output is written once.  A group of 32..256 columns is then
// 4..32 neighbouring lanes of one wave, so its largest magnitude needs no LDS.
// Magnitudes are compared as the bits of |v|: unsigned order is the order of
// the values, with infinity above every finite value and NaN above infinity,
// so a NaN is not lost as it is by a floating maximum.
//
// Measured (GPU time per call in a graph, one MI355X; a large copy reaches 5.2
// TB/s, an empty launch 1.8-2.0 us): rms_norm 8192x4096 bf16 onto bf16, e4m3 out
// 44.6 us (5.3 TB/s), 8192x4096 fp16 48.4-49.3 us (5.4-5.5 TB/s), 32768x128 5.0 us, one row
// of 4096 2.9 us; silu_mul 2048x12288 fp16 27.8 us (5.4 TB/s), to int8 with one
// scale per row 26.2 us, one row of 12288 fp32 2.7 us (group scales; 3.8 with one
// scale, where one workgroup does the row).

#include "common.h"

namespace lvq {

constexpr int kChunk = 8;          // columns a thread owns at a time
constexpr int kNone = 3;           // "no residual" beside LVQ_F32, LVQ_F16, LVQ_BF16
constexpr int kMaxCols = 65536;     // of any row
constexpr int kMaxRowCols = 32768;  // of a row that one workgroup holds in registers
constexpr int kRowThreads = 1024;

// ---------------------------------------------------------------- loads and stores

__device__ __forceinline__ float half_bits(uint32_t b) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}
__device__ __forceinline__ float bf16_bits(uint32_t b) {
  return __builtin_bit_cast(float, b << 16);
}
__device__ __forceinline__ uint32_t to_half_bits(float f) {
  return __builtin_bit_cast(uint16_t, (_Float16)f);
}
__device__ __forceinline__ uint32_t to_bf16_bits(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

template <int T>
struct Chunk {  // 8 values as they lie in memory
  uint4 q[T == LVQ_F32 ? 2 : 1];
};

// The column index through an empty statement, so that what the rare chunk at
// a row's end compares is formed there and not held in registers from the start.
__device__ __forceinline__ int opaque(int c) {
  asm volatile("" : "+v"(c));
  return c;
}

// Columns c..c+7 of a row; columns past cols read as 0.  A whole chunk is read
// 16 bytes at a time whatever its alignment (global memory takes any); the
// chunk that cols cuts reads its values one by one, the missing ones as copies
// of the last, so there is no branch per value.
template <int T>
__device__ __forceinline__ Chunk<T> load_chunk(const void* row, int c, int cols) {
  constexpr int E = T == LVQ_F32 ? 4 : 2;
  Chunk<T> r;
  if (c + kChunk <= cols) {
    __builtin_memcpy(&r, (const uint8_t*)row + (size_t)c * E, sizeof(r));
    return r;
  }
  uint32_t w[T == LVQ_F32 ? 8 : 4];
#pragma unroll
  for (int i = 0; i < (T == LVQ_F32 ? 8 : 4); ++i) w[i] = 0;
  if (c < cols) {
    c = opaque(c);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const int at = c + i < cols ? c + i : cols - 1;
      uint32_t v = T == LVQ_F32 ? ((const uint32_t*)row)[at] : ((const uint16_t*)row)[at];
      v = c + i < cols ? v : 0u;
      if constexpr (T == LVQ_F32) w[i] = v;
      else w[i >> 1] |= v << (16 * (i & 1));
    }
  }
  r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
  if constexpr (T == LVQ_F32) r.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  return r;
}

template <int T>
__device__ __forceinline__ void unpack(const Chunk<T>& r, float (&v)[kChunk]) {
#pragma unroll
  for (int h = 0; h < (T == LVQ_F32 ? 2 : 1); ++h) {
    const uint32_t w[4] = {r.q[h].x, r.q[h].y, r.q[h].z, r.q[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == LVQ_F32) {
        v[4 * h + i] = __builtin_bit_cast(float, w[i]);
      } else if constexpr (T == LVQ_F16) {
        v[2 * i] = half_bits(w[i] & 0xFFFFu);
        v[2 * i + 1] = half_bits(w[i] >> 16);
      } else {
        v[2 * i] = bf16_bits(w[i] & 0xFFFFu);
        v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
      }
    }
  }
}

// Columns c..c+7 (c < cols) of a row of `type` (fp32, fp16 or bf16) from fp32,
// rounded once to the nearest even.
__device__ __forceinline__ void store_chunk(void* row, int type, int c, int cols,
                                            const float (&v)[kChunk]) {
  if (type == LVQ_F32) {
    float* p = (float*)row + c;
    if (c + kChunk <= cols) {
      __builtin_memcpy(p, v, sizeof(v));
    } else {
      c = opaque(c);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (c + i < cols) p[i] = v[i];
    }
    return;
  }
  uint32_t b[4];
  if (type == LVQ_F16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = to_half_bits(v[2 * i]) | to_half_bits(v[2 * i + 1]) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = to_bf16_bits(v[2 * i]) | to_bf16_bits(v[2 * i + 1]) << 16;
  }
  uint16_t* p = (uint16_t*)row + c;
  if (c + kChunk <= cols) {
    __builtin_memcpy(p, b, sizeof(b));
  } else {
    c = opaque(c);
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (c + i < cols) p[i] = (uint16_t)(b[i >> 1] >> (16 * (i & 1)));
  }
}

// ---------------------------------------------------------------- maxima

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  // max of v and the value DPP routes to this lane (0 where the row is masked)
  const uint32_t m =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false);
  return v > m ? v : m;
}

// Sum and maximum over each aligned group of L = 16, 32 or 64 lanes, in all of
// them: quad swaps and mirrors inside a row of 16, then rows swapped pairwise.
// Every step adds the same two values on both sides, so all lanes get the same
// bits.
__device__ __forceinline__ uint32_t swap16(uint32_t v, uint32_t* other) {
  auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  *other = p[1];
  return p[0];
}
__device__ __forceinline__ uint32_t swap32(uint32_t v, uint32_t* other) {
  auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  *other = p[1];
  return p[0];
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_add<0xB1, 0xF>(v);
  v = dpp_add<0x4E, 0xF>(v);
  v = dpp_add<0x141, 0xF>(v);
  v = dpp_add<0x140, 0xF>(v);
  uint32_t o;
  if constexpr (L >= 32) {
    v = __builtin_bit_cast(float, swap16(__builtin_bit_cast(uint32_t, v), &o));
    v += __builtin_bit_cast(float, o);
  }
  if constexpr (L >= 64) {
    v = __builtin_bit_cast(float, swap32(__builtin_bit_cast(uint32_t, v), &o));
    v += __builtin_bit_cast(float, o);
  }
  return v;
}

template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = dpp_max<0xB1, 0xF>(v);
  v = dpp_max<0x4E, 0xF>(v);
  v = dpp_max<0x141, 0xF>(v);
  v = dpp_max<0x140, 0xF>(v);
  uint32_t o;
  if constexpr (L >= 32) {
    v = swap16(v, &o);
    v = v > o ? v : o;
  }
  if constexpr (L >= 64) {
    v = swap32(v, &o);
    v = v > o ? v : o;
  }
  return v;
}

// Maximum over the aligned group of `lanes` (4, 8, 16 or 32) lanes.
__device__ __forceinline__ uint32_t group_max(uint32_t v, int lanes) {
  v = dpp_max<0xB1, 0xF>(v);
  v = dpp_max<0x4E, 0xF>(v);
  if (lanes >= 8) v = dpp_max<0x141, 0xF>(v);
  if (lanes >= 16) v = dpp_max<0x140, 0xF>(v);
  if (lanes >= 32) {
    uint32_t o;
    v = swap16(v, &o);
    v = v > o ? v : o;
  }
  return v;
}

// ---------------------------------------------------------------- outputs

struct Out {
  void* out;
  float* scale;
  int cols;
  uint16_t type, group;
};

// Writes a row's results o[k] (columns 8 (t + k n) .. + 7 belong to thread t of
// the n that share the row); cols: a.cols, or 0 in lanes without a row.  LANES:
// the n are 16, 32 or 64 lanes of a wave; 0: a workgroup.  red: LDS words, one
// per wave of the workgroup, not in use by any thread.
template <int NV, int LANES>
__device__ __forceinline__ void emit(const Out& a, size_t row, const float (&o)[NV][kChunk], int t,
                                     int n, int cols, uint32_t* red) {
  if (a.type == LVQ_F16) {
    uint16_t* p = (uint16_t*)a.out + row * a.cols;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * n) * kChunk;
      if (c < cols) store_chunk(p, LVQ_F16, c, cols, o[k]);
    }
    return;
  }
  uint32_t top[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    top[k] = 0;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const uint32_t b = __builtin_bit_cast(uint32_t, o[k][i]) & 0x7FFFFFFFu;
      top[k] = top[k] > b ? top[k] : b;
    }
  }
  if (a.group == 0) {
    uint32_t m = top[0];
#pragma unroll
    for (int k = 1; k < NV; ++k) m = m > top[k] ? m : top[k];
    m = lanes_max<LANES ? LANES : kWave>(m);
    if constexpr (LANES == 0) {
      if ((t & (kWave - 1)) == 0) red[t / kWave] = m;
      __syncthreads();
      m = red[0];
      for (int w = 1; w < n / kWave; ++w) m = m > red[w] ? m : red[w];
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) top[k] = m;
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) top[k] = group_max(top[k], a.group / kChunk);
  }
  const float most = a.type == LVQ_I8 ? 127.f : 448.f;
  uint8_t* p = (uint8_t*)a.out + row * a.cols;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * n) * kChunk;
    if (c >= cols) continue;
    const float m = __builtin_bit_cast(float, top[k]);
    // below 2^-100 the reciprocal leaves the fp32 range; NaN compares false
    const bool ok = top[k] < 0x7F800000u && m >= 0x1p-100f;
    const float inv = ok ? most / m : 0.f;
    if (a.group == 0 ? c == 0 : (c & (a.group - 1)) == 0)
      a.scale[a.group == 0 ? row : row * ((a.cols + a.group - 1) / a.group) + c / a.group] =
          ok ? m / most : top[k] < 0x7F800000u ? 0.f : m;
    uint32_t lo = 0, hi = 0;
    float v[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = ok ? o[k][i] * inv : 0.f;
    if (a.type == LVQ_I8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo |= ((uint32_t)(int)__builtin_rintf(v[i]) & 0xFFu) << (8 * i);
        hi |= ((uint32_t)(int)__builtin_rintf(v[i + 4]) & 0xFFu) << (8 * i);
      }
    } else {
      int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
      lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], q, true);
      q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
      hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], q, true);
    }
    if (c + kChunk <= cols) {
      const uint32_t q[2] = {lo, hi};
      __builtin_memcpy(p + c, q, sizeof(q));
    } else {
      const int e = opaque(c);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (e + i < cols) p[e + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
    if constexpr (NV > 2) __builtin_amdgcn_sched_barrier(0);
  }
}

// ---------------------------------------------------------------- rms_norm

// The kernels' arguments are under 128 bytes, the launch's own dimensions among
// them (read through the language's variables they bring 200 bytes of hidden
// arguments along): in a plain program a launch with 112 bytes of arguments costs
// the host 2.9 us, one with 128 or more 3.6.
struct NormArgs {
  const void* x;
  int64_t x_stride;  // bytes
  const void* residual;
  void* residual_out;
  const void* weight;
  float eps;
  int rows, grid;
  uint16_t residual_type, weight_type, threads;
  Out out;
};
static_assert(sizeof(NormArgs) <= 112, "launches of 128 bytes and more are slower");

__device__ __forceinline__ void load_weight(const NormArgs& a, int c, float (&w)[kChunk]) {
  if (!a.weight) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) w[i] = 1.f;
  } else if (a.weight_type == LVQ_F32) {
    unpack(load_chunk<LVQ_F32>(a.weight, c, a.out.cols), w);
  } else if (a.weight_type == LVQ_F16) {
    unpack(load_chunk<LVQ_F16>(a.weight, c, a.out.cols), w);
  } else {
    unpack(load_chunk<LVQ_BF16>(a.weight, c, a.out.cols), w);
  }
}

// A row per workgroup, or per 16, 32 or 64 lanes of a wave where they hold one
// (LANES).  Rows are taken a grid apart.
template <int TX, int TR, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? 256 : kRowThreads) rms_norm_kernel(NormArgs a) {
  __shared__ uint32_t red[2][2][kRowThreads / kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = a.threads / kWave;
  constexpr int kRows = LANES ? kWave / LANES : 1;  // of a wave
  const int t = LANES ? lane % LANES : (int)threadIdx.x;
  const int n = LANES ? LANES : (int)a.threads;
  const int64_t step = LANES ? (int64_t)a.grid * nw * kRows : a.grid;
  constexpr int kResBytes = TR == LVQ_F32 ? 4 : 2;
  // up to two chunks per thread: the weights are read once, ahead of the rows
  // (they are the same columns of every row); more would not fit beside the row
  float wt[NV][kChunk];
  if constexpr (NV <= 2) {
#pragma unroll
    for (int k = 0; k < NV; ++k) load_weight(a, (t + k * n) * kChunk, wt[k]);
  }
  int turn = 0;
  for (int64_t row0 = LANES ? ((int64_t)blockIdx.x * nw + wv) * kRows : blockIdx.x;
       row0 < a.rows; row0 += step, turn ^= 1) {
    const int64_t row = LANES ? row0 + lane / (LANES ? LANES : 1) : row0;
    const int cols = kRows == 1 || row < a.rows ? a.out.cols : 0;  // 0: these lanes have no row
    const uint8_t* xr = (const uint8_t*)a.x + row * a.x_stride;
    const uint8_t* rr = (const uint8_t*)a.residual + (size_t)row * a.out.cols * kResBytes;
    // up to two chunks per thread: every load goes out before the first is
    // used; more: two at a time, or the raw values would not fit in registers
    constexpr int G = NV < 2 ? NV : 2;
    float h[NV][kChunk], part = 0.f;
#pragma unroll
    for (int k0 = 0; k0 < NV; k0 += G) {
      Chunk<TX> xc[G];
      Chunk<TR == kNone ? LVQ_F16 : TR> rc[G];
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int c = (t + (k0 + k) * n) * kChunk;
        xc[k] = load_chunk<TX>(xr, c, cols);
        if constexpr (TR != kNone) rc[k] = load_chunk<TR>(rr, c, cols);
      }
#pragma unroll
      for (int k = 0; k < G; ++k) {
        unpack(xc[k], h[k0 + k]);
        if constexpr (TR != kNone) {
          float r[kChunk];
          unpack(rc[k], r);
#pragma unroll
          for (int i = 0; i < kChunk; ++i) h[k0 + k][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          part = __builtin_fmaf(h[k0 + k][i], h[k0 + k][i], part);
      }
      if constexpr (NV > 2) __builtin_amdgcn_sched_barrier(0);
    }
    if (a.residual_out) {
      uint8_t* ro = (uint8_t*)a.residual_out +
                    (size_t)row * a.out.cols * (a.residual_type == LVQ_F32 ? 4 : 2);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (t + k * n) * kChunk;
        if (c < cols) store_chunk(ro, a.residual_type, c, cols, h[k]);
        if constexpr (NV > 2) __builtin_amdgcn_sched_barrier(0);
      }
    }
    float sum = lanes_sum<LANES ? LANES : kWave>(part);
    if constexpr (LANES == 0) {
      // two sets of LDS words, used in turn: a wave can be at most one barrier
      // ahead of another, so it never writes a set that is still being read
      float* rs = (float*)red[turn][0];
      if (lane == 0) rs[wv] = sum;
      __syncthreads();
      sum = rs[0];
      for (int w = 1; w < nw; ++w) sum += rs[w];
    }
    const float inv = rsqrtf(sum / (float)a.out.cols + a.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (NV > 2) load_weight(a, (t + k * n) * kChunk, wt[k]);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) h[k][i] = h[k][i] * inv * wt[k][i];
      if constexpr (NV > 2) __builtin_amdgcn_sched_barrier(0);
    }
    emit<NV, LANES>(a.out, (size_t)row, h, t, n, cols, red[turn][1]);
  }
}

// Lanes or threads that share a row and chunks per thread.  Up to 512 columns 16,
// 32 or 64 lanes; above, a workgroup with one chunk per thread for few rows (the
// shortest way through one row), two for many (fewer waves meet at a row's
// barriers and each has more loads in flight: 2048x8192 int8 25.5 us with 512
// threads and two chunks, 36.7 with 1024 and one, 29.1 with 256 and four;
// 8192x4096 44.6 with two, 45.0 with one), four where 1024 threads need them.
struct RowShape {
  int nv, threads, lanes;
};
RowShape row_shape(int rows, int cols, int group) {
  const int chunks = (cols + kChunk - 1) / kChunk;
  if (chunks <= kWave)  // a row's lanes hold whole groups: 256 columns are 32 lanes
    return {1, 256, chunks <= 16 && group <= 128 ? 16 : chunks <= 32 ? 32 : 64};
  const int nv = chunks > 2 * kRowThreads ? 4
                 : chunks > kRowThreads || (rows >= device_cus() && chunks > 256) ? 2 : 1;
  return {nv, ((chunks + nv - 1) / nv + kWave - 1) / kWave * kWave, 0};
}

// As many workgroups as the chip holds at once where lanes share a row, four times
// that where a workgroup does, so that those which end early are followed by others
// (8192x4096: 44.6 us with four times, 47.2 with once).  With lanes the smaller grid
// reads the weights less often: 70000x64 fp16 6.5 us with once, 7.7 with four times;
// far longer inputs lose by it, 131072x512 fp16 49.0 against 47.5, 1000000x64 to int8
// 131 against 104.
int row_grid(int rows, const RowShape& s) {
  const int per = s.lanes ? s.threads / s.lanes : 1;
  const long long wgs = ((long long)rows + per - 1) / per;
  const long long most = (long long)device_cus() * (2048 / s.threads) * (s.lanes ? 1 : 4);
  return (int)(wgs < most ? wgs : most);
}

template <int TX, int TR>
int launch_norm_row(NormArgs a, hipStream_t st) {
  const RowShape s = row_shape(a.rows, a.out.cols, a.out.group);
  a.grid = row_grid(a.rows, s), a.threads = (uint16_t)s.threads;
  const dim3 grid(a.grid), block(s.threads);
  clear_hip_error();
  if (s.lanes == 16) hipLaunchKernelGGL((rms_norm_kernel<TX, TR, 1, 16>), grid, block, 0, st, a);
  else if (s.lanes == 32) hipLaunchKernelGGL((rms_norm_kernel<TX, TR, 1, 32>), grid, block, 0, st, a);
  else if (s.lanes == 64) hipLaunchKernelGGL((rms_norm_kernel<TX, TR, 1, 64>), grid, block, 0, st, a);
  else if (s.nv == 1) hipLaunchKernelGGL((rms_norm_kernel<TX, TR, 1, 0>), grid, block, 0, st, a);
  else if (s.nv == 2) hipLaunchKernelGGL((rms_norm_kernel<TX, TR, 2, 0>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((rms_norm_kernel<TX, TR, 4, 0>), grid, block, 0, st, a);
  return launch_status();
}

template <int TX>
int launch_norm(const NormArgs& a, hipStream_t st) {
  if (!a.residual) return launch_norm_row<TX, kNone>(a, st);
  if (a.residual_type == LVQ_F32) return launch_norm_row<TX, LVQ_F32>(a, st);
  if (a.residual_type == LVQ_F16) return launch_norm_row<TX, LVQ_F16>(a, st);
  return launch_norm_row<TX, LVQ_BF16>(a, st);
}

// ---------------------------------------------------------------- silu_mul

struct SiluArgs {
  const void *gate, *up;
  int64_t stride;  // bytes
  int rows, grid, segs;
  uint16_t seg_shift, threads;
  Out out;
};
static_assert(sizeof(SiluArgs) <= 112, "launches of 128 bytes and more are slower");

template <int T>
__device__ __forceinline__ void silu_chunk(const Chunk<T>& gc, const Chunk<T>& uc,
                                           float (&o)[kChunk]) {
  float g[kChunk], u[kChunk];
  unpack(gc, g);
  unpack(uc, u);
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    // e^-g as 2^(-g log2 e); both of the hardware's approximations (2^v and
    // 1/v) are within an ulp, the product of the exponent off by up to 2 |g| 2^-24 of
    // the power, which an 11-bit output hides.  The hardware's 1/v is 0 where it
    // would be subnormal (g below -87.3), so a quarter of 1 + e^-g is inverted and a
    // quarter of g multiplied: right down to where e^-g leaves fp32 (g below
    // -88.72, then 0).
    const float e = __builtin_amdgcn_exp2f(g[i] * -1.44269504f);
    o[i] = g[i] * 0.25f * __builtin_amdgcn_rcpf(__builtin_fmaf(e, 0.25f, 0.25f)) * u[i];
  }
}

// One scale per row: a row per workgroup or per 16, 32 or 64 lanes.
template <int T, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? 256 : kRowThreads) silu_row_kernel(SiluArgs a) {
  __shared__ uint32_t red[2][kRowThreads / kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = a.threads / kWave;
  constexpr int kRows = LANES ? kWave / LANES : 1;  // of a wave
  const int t = LANES ? lane % LANES : (int)threadIdx.x;
  const int n = LANES ? LANES : (int)a.threads;
  const int64_t step = LANES ? (int64_t)a.grid * nw * kRows : a.grid;
  int turn = 0;
  for (int64_t row0 = LANES ? ((int64_t)blockIdx.x * nw + wv) * kRows : blockIdx.x;
       row0 < a.rows; row0 += step, turn ^= 1) {
    const int64_t row = LANES ? row0 + lane / (LANES ? LANES : 1) : row0;
    const int cols = kRows == 1 || row < a.rows ? a.out.cols : 0;  // 0: these lanes have no row
    const uint8_t* gr = (const uint8_t*)a.gate + row * a.stride;
    const uint8_t* ur = (const uint8_t*)a.up + row * a.stride;
    Chunk<T> gc[NV], uc[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * n) * kChunk;
      gc[k] = load_chunk<T>(gr, c, cols);
      uc[k] = load_chunk<T>(ur, c, cols);
    }
    float o[NV][kChunk];
#pragma unroll
    for (int k = 0; k < NV; ++k) silu_chunk<T>(gc[k], uc[k], o[k]);
    emit<NV, LANES>(a.out, (size_t)row, o, t, n, cols, red[turn]);
  }
}

// Chunks are independent (fp16, or groups inside a wave): a workgroup takes 256
// chunks, 2^seg_shift neighbours of each of 256 >> seg_shift rows.
template <int T>
__global__ void __launch_bounds__(256) silu_flat_kernel(SiluArgs a) {
  const int seg = 1 << a.seg_shift, per = 256 >> a.seg_shift;
  const int64_t tiles = ((int64_t)a.rows + per - 1) / per * a.segs;
  for (int64_t i = blockIdx.x; i < tiles; i += a.grid) {
    const int64_t block = i / a.segs;
    const int64_t row = block * per + (threadIdx.x >> a.seg_shift);
    const int chunk = (int)(i - block * a.segs) * seg + (threadIdx.x & (seg - 1));
    const int c = chunk * kChunk, cols = row < a.rows ? a.out.cols : 0;  // 0: no row here
    const uint8_t* gr = (const uint8_t*)a.gate + row * a.stride;
    const uint8_t* ur = (const uint8_t*)a.up + row * a.stride;
    float o[1][kChunk];
    silu_chunk<T>(load_chunk<T>(gr, c, cols), load_chunk<T>(ur, c, cols), o[0]);
    emit<1, kWave>(a.out, (size_t)row, o, chunk, 0, cols, nullptr);
  }
}

template <int T>
int launch_silu(SiluArgs& a, hipStream_t st) {
  clear_hip_error();
  if (a.out.type != LVQ_F16 && a.out.group == 0) {
    const RowShape s = row_shape(a.rows, a.out.cols, a.out.group);
    a.grid = row_grid(a.rows, s), a.threads = (uint16_t)s.threads;
    const dim3 grid(a.grid), block(s.threads);
    if (s.lanes == 16) hipLaunchKernelGGL((silu_row_kernel<T, 1, 16>), grid, block, 0, st, a);
    else if (s.lanes == 32) hipLaunchKernelGGL((silu_row_kernel<T, 1, 32>), grid, block, 0, st, a);
    else if (s.lanes == 64) hipLaunchKernelGGL((silu_row_kernel<T, 1, 64>), grid, block, 0, st, a);
    else if (s.nv == 1) hipLaunchKernelGGL((silu_row_kernel<T, 1, 0>), grid, block, 0, st, a);
    else if (s.nv == 2) hipLaunchKernelGGL((silu_row_kernel<T, 2, 0>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((silu_row_kernel<T, 4, 0>), grid, block, 0, st, a);
    return launch_status();
  }
  const int chunks = (a.out.cols + kChunk - 1) / kChunk;
  a.seg_shift = 5;  // at least the 32 lanes of the widest group
  while (a.seg_shift < 8 && (1 << a.seg_shift) < chunks) ++a.seg_shift;
  a.segs = (chunks + (1 << a.seg_shift) - 1) >> a.seg_shift;
  const int per = 256 >> a.seg_shift;
  const long long tiles = ((long long)a.rows + per - 1) / per * a.segs;
  const long long most = (long long)device_cus() * 32;
  a.grid = (int)(tiles < most ? tiles : most), a.threads = 256;
  hipLaunchKernelGGL(silu_flat_kernel<T>, dim3(a.grid), dim3(256), 0, st, a);
  return launch_status();
}

// ---------------------------------------------------------------- checks

inline bool float_type(int t) { return t == LVQ_F32 || t == LVQ_F16 || t == LVQ_BF16; }
inline size_t type_bytes(int t) { return t == LVQ_F32 ? 4 : t == LVQ_I8 || t == LVQ_E4M3 ? 1 : 2; }
inline bool aligned_to(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

// Scales per row of 8-bit outputs.
inline int scale_count(const Out& o) { return o.group ? (o.cols + o.group - 1) / o.group : 1; }

// The output arguments both entry points share; fills *o.
int check_out(void* out, int out_type, float* out_scale, int out_group, int rows, int cols,
              Out* o) {
  if (out_type != LVQ_F16 && out_type != LVQ_I8 && out_type != LVQ_E4M3) return LVQ_E_SHAPE;
  const bool eight = out_type != LVQ_F16;
  if (out_group != 0 &&
      (!eight || (out_group != 32 && out_group != 64 && out_group != 128 && out_group != 256)))
    return LVQ_E_SHAPE;
  if (!eight && out_scale) return LVQ_E_SHAPE;
  if (rows && cols && (!out || (eight && !out_scale))) return LVQ_E_NULL;
  if (!aligned16(out) || !aligned16(out_scale)) return LVQ_E_ALIGN;
  o->out = out, o->scale = out_scale, o->cols = cols;
  o->type = (uint16_t)out_type, o->group = (uint16_t)out_group;
  return LVQ_OK;
}

// Whether `rows` rows `stride` values apart (stride >= cols) can be addressed.
inline bool stride_ok(int rows, int64_t stride) {
  return stride <= (INT64_MAX >> 4) / (rows > 0 ? rows : 1);
}

struct Range {
  const void* p;
  size_t n;
};
// Bytes from the first to the last value of `rows` strided rows.
inline size_t strided_bytes(int rows, int cols, int64_t stride, int type) {
  return ((size_t)(rows - 1) * stride + cols) * type_bytes(type);
}

}  // namespace lvq

using namespace lvq;

extern "C" int lvq_rms_norm(const void* x, int x_type, int64_t x_stride, const void* residual,
                            int residual_type, void* residual_out, const void* weight,
                            int weight_type, float eps, int rows, int cols, void* out,
                            int out_type, float* out_scale, int out_group, void* stream) {
  if (rows < 0 || cols < 0 || cols > kMaxRowCols || x_stride < cols || !stride_ok(rows, x_stride))
    return LVQ_E_SHAPE;
  if (!float_type(x_type) || ((residual || residual_out) && !float_type(residual_type)) ||
      (weight && !float_type(weight_type)))
    return LVQ_E_SHAPE;
  NormArgs a;
  const int e = check_out(out, out_type, out_scale, out_group, rows, cols, &a.out);
  if (e) return e;
  if (rows == 0 || cols == 0) return LVQ_OK;
  if (!x) return LVQ_E_NULL;
  if (!aligned_to(x, type_bytes(x_type)) || !aligned16(residual) || !aligned16(residual_out) ||
      !aligned16(weight))
    return LVQ_E_ALIGN;
  const size_t all = (size_t)rows * cols;
  const Range in[3] = {{x, strided_bytes(rows, cols, x_stride, x_type)},
                       {residual, residual ? all * type_bytes(residual_type) : 0},
                       {weight, weight ? (size_t)cols * type_bytes(weight_type) : 0}};
  const Range made[3] = {{residual_out, residual_out ? all * type_bytes(residual_type) : 0},
                         {out, all * type_bytes(out_type)},
                         {out_scale, out_scale ? (size_t)rows * scale_count(a.out) * 4 : 0}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 3; ++j) {
      const bool same_stream = i == 0 && j == 1 && residual == residual_out;
      if (!same_stream && ranges_overlap(made[i].p, made[i].n, in[j].p, in[j].n))
        return LVQ_E_SHAPE;
      if (j > i && ranges_overlap(made[i].p, made[i].n, made[j].p, made[j].n)) return LVQ_E_SHAPE;
    }
  }
  a.x = x, a.x_stride = x_stride * (int64_t)type_bytes(x_type);
  a.residual = residual, a.residual_out = residual_out;
  a.residual_type = (uint16_t)residual_type, a.weight = weight;
  a.weight_type = (uint16_t)weight_type, a.eps = eps, a.rows = rows;
  hipStream_t st = (hipStream_t)stream;
  if (x_type == LVQ_F32) return launch_norm<LVQ_F32>(a, st);
  if (x_type == LVQ_F16) return launch_norm<LVQ_F16>(a, st);
  return launch_norm<LVQ_BF16>(a, st);
}

extern "C" int lvq_silu_mul(const void* gate, const void* up, int in_type, int64_t in_stride,
                            int rows, int cols, void* out, int out_type, float* out_scale,
                            int out_group, void* stream) {
  if (rows < 0 || cols < 0 || cols > kMaxCols || in_stride < cols ||
      !stride_ok(rows, in_stride) || !float_type(in_type))
    return LVQ_E_SHAPE;
  if (cols > kMaxRowCols && out_type != LVQ_F16 && out_group == 0) return LVQ_E_SHAPE;
  SiluArgs a;
  const int e = check_out(out, out_type, out_scale, out_group, rows, cols, &a.out);
  if (e) return e;
  if (rows == 0 || cols == 0) return LVQ_OK;
  if (!gate || !up) return LVQ_E_NULL;
  const size_t tb = type_bytes(in_type);
  if (!aligned_to(gate, tb) || !aligned_to(up, tb)) return LVQ_E_ALIGN;
  const size_t in_bytes = strided_bytes(rows, cols, in_stride, in_type);
  const Range in[2] = {{gate, in_bytes}, {up, in_bytes}};
  const Range made[2] = {{out, (size_t)rows * cols * type_bytes(out_type)},
                         {out_scale, out_scale ? (size_t)rows * scale_count(a.out) * 4 : 0}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (ranges_overlap(made[i].p, made[i].n, in[j].p, in[j].n)) return LVQ_E_SHAPE;
  if (ranges_overlap(made[0].p, made[0].n, made[1].p, made[1].n)) return LVQ_E_SHAPE;
  a.gate = gate, a.up = up, a.stride = in_stride * (int64_t)tb;
  a.rows = rows, a.seg_shift = 8, a.segs = 1;
  hipStream_t st = (hipStream_t)stream;
  if (in_type == LVQ_F32) return launch_silu<LVQ_F32>(a, st);
  if (in_type == LVQ_F16) return launch_silu<LVQ_F16>(a, st);
  return launch_silu<LVQ_BF16>(a, st);
}
