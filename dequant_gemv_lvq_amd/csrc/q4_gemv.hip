// 4-bit matvec with group scales (q4_gemv, q4_gemv_q8).
//
//   y[b][r] = sum_u s_ru (sum_(c in u) q_rc x_bc - z_ru sum_(c in u) x_bc)
//
// over the units u of 32 columns (16 bytes of codes), inside which scale and
// zero are constant.  The inner sums run on the matrix cores: the 4x4x4 MFMA in
// 16 blocks multiplies, per instruction, 16 independent 4 (batch) x 4 (columns)
// by 4 (columns) x 4 (rows) products, which is the shape of a matvec of up to
// four batch rows.  Lane l holds row l % 4 of a quad of rows and unit l / 4 of
// a step of 16 units: its 16 bytes of codes are its own B operands, the x of
// its unit (batch row l % 4) its A operands, and the result leaves in lane l the
// four batch sums of its own row and unit, so scale and zero are applied in the
// lane that loaded them, in fp32, once per unit.
//
// No conversion of the codes to floats: a 4-bit value inside the ten mantissa bits
// of an fp16 is a subnormal, the value times a power of two.  Shifts and masks give
// two operands per 8 codes (columns 0, 4, 2, 6 and 1, 5, 3, 7 of the eight; x is
// stored in LDS in that order).  The position matters: the matrix core aligns a
// product by the exponents as stored, as if the code were as large as the top of
// the ten bits, so what a code lies below it is lost at the lower end of the sum.
//   fp16 x   bits 6..9 (eight operations per 8 codes): the sum q x0 + q x1 keeps
//            every x1 down to 2^-20 x0, as fp32 does for a 4-bit q.  In bits 4..7
//            (seven operations) it kept them to 2^-18, and the error against 64
//            bits rose above an fp32 product's where codes lie close to their zero
//            and x has outliers: norms of 0.9e-6 to 1.8e-6 of the result's at 4096
//            columns, 1.2e-7 to 3.4e-7 now; an fp32 product of unpacked weights has
//            4.6e-7 to 5.6e-7.  It takes 0 to 2 % of the time of the shapes below.
//   e4m3 x   bits 4..7: x itself spans 2^-17 of its largest value at most, so
//            nothing is lost (0.4e-7 to 0.9e-7, whatever the codes).
//   int8 x   two masks and a shift give the codes as bytes, and the sums are exact
//            32-bit integers.
// The sum starts from minus zero times the unit's sum of x: where x has one sign and
// the codes lie close to a zero far from 0 the two cancel, as the order of the sum
// in fp32 has it (13..15 about zero 14, x > 0: 1.4e-6).
//
// The weights are the bytes (4.1 to 5 bits each): 4 flops per byte at batch 1.
// Each wave streams 1 KiB of codes per step (4 rows x 256 contiguous bytes) in
// chunks of four, two chunks in flight; x and the sums of x over every unit sit
// in LDS.  Loads are counted: one of 64 lanes takes a CU's load unit 16 cycles
// whatever it returns, so the scales and zeros of four steps come with one load
// each (16 groups x 4 rows, or 16 x 2 bytes a row) and reach their lanes through
// ds_bpermute.  A chunk ends with its quad, so the last one of a quad costs four
// loads of codes whatever steps it holds: rows of up to 1024 columns run below the
// memory's rate for that (70003x96 10.4 us).
//
// Measured (GPU time per call in a graph over rotating matrices, one MI355X; a
// plain read of that many bytes runs at up to 6.4 TB/s, an empty launch 1.8 us):
// 131072x4096 batch 1 45-47 us, 5.9-6.1 TB/s, bound by that read; 4096x12288
// batch 1 7.4-7.9 us, 12288x4096 7.1-7.4 us (3.3-3.5 and 3.5-3.7 TB/s); 4096x12288
// batch 4 9.7-10.7 us, where each CU brings in 96 KiB of x; 4096x4096 3.8-4.4 us,
// 1024x4096 3.3 us, bound by the launch and two round trips to memory.  With the
// codes taken as they are, not unpacked (a timing variant), 131072x4096 took 43.6 us
// instead of 45.3, 12288x4096 6.3 instead of 7.1, 4096x12288 batch 4 9.0 instead of
// 9.8; without the loads of x the last took 9.2, without ordering and summing x 9.8.
// A full chunk's block holds 43-44 vector instructions per step at batch 1, 32 of
// them unpack the codes and 8 are matrix products, and 6 LDS reads.

#include <type_traits>

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

// What a call hands to the launch.
struct Q4Call {
  const uint8_t* codes;
  const uint16_t* scale;
  const uint16_t* zero;
  int gshift, rows, cols;
  const void* x;
  const float* xscale;
  int xshift;
  float* y;
  int batch;
};

// The kernel's arguments: under 128 bytes, and the launch's own dimensions among
// them (read through the language's variables they bring 200 bytes of hidden
// arguments along).  In a plain program a launch with 112 bytes of arguments
// costs the host 2.9 us, one with 128 or more 3.6.
struct Q4Args {
  const uint8_t* codes;
  const uint16_t* scale;
  const uint16_t* zero;
  const void* x;
  const float* xscale;
  float* y;
  int rows, cols, nunits, steps, groups, waves;
  uint8_t gshift, xshift;
  uint16_t batch;
  // how a workgroup's quads are dealt: whole ones per wave and divided steps per
  // wave, [0] in the first `extra` workgroups, which have quads + 1, [1] in the others
  int wgs, extra, quads, whole[2];
  uint16_t per[2];
};
static_assert(sizeof(Q4Args) <= 112, "launches of 128 bytes and more are slower");

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

// The bit of an fp16 subnormal where a code starts, and what that bit is worth.
constexpr int code_bit(int X) { return X == kQ4F16 ? 6 : 4; }
constexpr float code_unit(int X) { return X == kQ4F16 ? 0x1p-18f : 0x1p-20f; }
constexpr int kQ4Waves = 16;   // waves per workgroup at most
constexpr int kStepUnits = 16; // units of 32 columns per step
constexpr int kChunk = 4;      // steps a wave loads at a time
constexpr int kXAhead = 6;     // pieces of x a wave requests at a time

// LDS: x, then per unit and batch row the sum of x (see put_x8), then (8-bit x)
// its scale, then a partial result per wave.
//
// x of a step: a slab of 16-byte pieces per word of a unit (f16; per pair of
// words for int8), unit by unit, batch rows together.  A wave reads a slab in
// one run; slabs are 16 bytes further apart than they are long, or the four
// lanes that write a unit's words would write the same banks.
constexpr int slab_bytes(int B) { return 256 * B + 16; }
constexpr int x_step_bytes(int B, int X) { return (X == kQ4I8 ? 2 : 4) * slab_bytes(B); }
constexpr size_t sum_step_bytes(int B) { return kStepUnits * (size_t)B * 4; }
inline size_t q4_lds_bytes(int B, int X, int steps) {
  return (size_t)steps * (x_step_bytes(B, X) + sum_step_bytes(B) * (X == kQ4F16 ? 1 : 2)) +
         kQ4Waves * 4 * (size_t)B * 4;
}

__device__ __forceinline__ float f16_to_f32(uint32_t b) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t q4_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

// ---------------------------------------------------------------- x into LDS

// Eight columns of a batch row as they lie in memory (16 bytes of fp16, or 8),
// zeros past the row's end.
//   load_x8    rows of a multiple of eight columns; rx: the row
//   whole_x8   rows that start anywhere (global memory takes any alignment):
//              zeros too for the eight that the row's end cuts
//   cut_x8     those, value by value, zeros in every other lane
template <int X>
__device__ __forceinline__ u32x4_t load_x8(__amdgpu_buffer_rsrc_t rx, int c) {
  if constexpr (X == kQ4F16) {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rx, c * 2, 0, 0));
  } else {
    const auto h = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rx, c, 0, 0));
    return u32x4_t{h.x, h.y, 0, 0};
  }
}

template <int X>
__device__ __forceinline__ u32x4_t whole_x8(const uint8_t* row, int c, int cols) {
  constexpr int E = X == kQ4F16 ? 2 : 1;
  u32x4_t v = {0, 0, 0, 0};
  if (c + 8 <= cols) __builtin_memcpy(&v, row + (size_t)c * E, 8 * E);
  return v;
}

template <int X>
__device__ __forceinline__ u32x4_t cut_x8(__amdgpu_buffer_rsrc_t rx, int c, int cols) {
  constexpr int E = X == kQ4F16 ? 2 : 1;
  u32x4_t v = {0, 0, 0, 0};
  const int past = ~(cols - 8 - c) & (int)0x80000000;  // set where all eight are inside
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = ((c + i) * E) | past;
    if constexpr (E == 2)
      v[i >> 1] |= (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rx, at, 0, 0)
                   << (16 * (i & 1));
    else
      v[i >> 2] |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rx, at, 0, 0)
                   << (8 * (i & 3));
  }
  return v;
}

// The pairs (x0, x4) (x2, x6) (x1, x5) (x3, x7) of eight fp16.
__device__ __forceinline__ u32x4_t pair_order(u32x4_t d) {
  return u32x4_t{__builtin_amdgcn_perm(d.z, d.x, 0x05040100u),
                 __builtin_amdgcn_perm(d.w, d.y, 0x05040100u),
                 __builtin_amdgcn_perm(d.z, d.x, 0x07060302u),
                 __builtin_amdgcn_perm(d.w, d.y, 0x07060302u)};
}

// Eight columns (word w of unit u of step t, batch row bb) into LDS, and, from
// the quad of lanes that holds a unit, minus the unit's sum (with zeros), or
// minus eight times it, as the matrix core's sum takes it, and its scale s.
template <int B, int X, bool Z>
__device__ __forceinline__ void put_x8(uint8_t* xs, float* sums, float* scaled,
                                       u32x4_t v, float s, int bb, int t, int lane) {
  const int ul = lane >> 2, w = lane & 3;
  float sum;
  if constexpr (X == kQ4I8) {
    // even and odd columns apart, as masking the codes' bytes leaves them
    const u32x2_t o = {__builtin_amdgcn_perm(v.y, v.x, 0x06040200u),
                       __builtin_amdgcn_perm(v.y, v.x, 0x07050301u)};
    *(u32x2_t*)(xs + t * x_step_bytes(B, X) + (w >> 1) * slab_bytes(B) + (ul * B + bb) * 16 +
                (w & 1) * 8) = o;
    const int s = __builtin_amdgcn_sdot4((int)v.x, 0x01010101, 0, false);
    sum = (float)__builtin_amdgcn_sdot4((int)v.y, 0x01010101, s, false);
  } else {
    u32x4_t h = v;
    if constexpr (X == kQ4E4M3) {  // every e4m3 value is an fp16 value
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], false);
        const float2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], true);
        h[2 * i] = __builtin_bit_cast(uint32_t, lvq_half2{(_Float16)lo.x, (_Float16)lo.y});
        h[2 * i + 1] = __builtin_bit_cast(uint32_t, lvq_half2{(_Float16)hi.x, (_Float16)hi.y});
      }
    }
    *(u32x4_t*)(xs + t * x_step_bytes(B, X) + w * slab_bytes(B) + (ul * B + bb) * 16) =
        pair_order(h);
    constexpr uint32_t kOnes = 0x3C003C00u;
    sum = dot2(h.x, kOnes, dot2(h.y, kOnes, dot2(h.z, kOnes, dot2(h.w, kOnes, 0.f))));
  }
  sum = dpp_add<0x4E, 0xF>(dpp_add<0xB1, 0xF>(sum));  // the quad's four words
  if (w == 0) {
    const int u = t * kStepUnits + ul, at = u * B + bb;
    sum *= (Z ? -1.f : -8.f) * (X == kQ4I8 ? 1.f : code_unit(X));
    if constexpr (X == kQ4I8 && !Z) sum = __builtin_bit_cast(float, (int)sum);  // a whole number
    sums[at] = sum;
    if constexpr (X != kQ4F16) scaled[at] = s;
  }
}

// ---------------------------------------------------------------- the kernel

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

// What a wave has in flight: four steps of codes and the scales (low half) and
// zeros (high half) of their groups, NS registers of them: 4 / NS steps share
// one, lane 4 k + r holding the k-th of up to 16 groups of row r.
template <int NS>
struct Q4Chunk {
  u32x4_t w[kChunk];
  uint16_t s[NS], z[NS];
};

// Quads of rows go round the workgroups, and a workgroup's go round its waves,
// so that the whole chip reads one window of neighbouring rows at a time (with a
// run of quads per wave, streams a large power of two apart, 131072x4096 took 48
// instead of 45 us); of the last round, the steps are dealt to the waves in
// equal contiguous parts.  A quad whose steps lie in more than one wave is
// joined in LDS at the end, in order, by the wave that holds its first step.
// RING: chunks of four steps in flight per wave, 1 where no wave has more.
template <int B, int X, int NS, bool Z, int RING>
__global__ void __launch_bounds__(kQ4Waves * kWave) q4_gemv_kernel(Q4Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int nunits = a.nunits, steps = a.steps, groups = a.groups;
  uint8_t* xs = smem;
  float* sums = (float*)(smem + steps * x_step_bytes(B, X));
  float* scaled = sums + steps * (sum_step_bytes(B) / 4);
  float* join = X == kQ4F16 ? scaled : scaled + steps * (sum_step_bytes(B) / 4);

  const int lane = threadIdx.x & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = a.waves;

  // 1. x: each wave takes pieces of 64 x 8 columns (one step of one batch row),
  //    kXAhead requested at a time; the weights' first loads go out behind the
  //    last of them, so the wait for x does not include the weights (with a
  //    first chunk of weights ahead of x 4096x12288 at batch 4 takes 11.6 us
  //    instead of 10.6, with both chunks 12.0)
  const int pieces = B * steps;  // of batch rows past the batch: zeros
  const int xgroups = groups_of(nunits, a.xshift);
  u32x4_t xv[kXAhead];
  float xsc[kXAhead];
  constexpr int E = X == kQ4F16 ? 2 : 1;
  const bool even = a.cols % 8 == 0;  // every row starts at a piece's alignment
  auto row_at = [&](int bb) { return (const uint8_t*)a.x + (size_t)bb * a.cols * E; };
  auto row_of = [&](int bb) { return q4_rsrc(row_at(bb), bb < a.batch ? a.cols * E : 0); };
  auto load_ahead = [&](int i0, auto is_even) {
#pragma unroll
    for (int k = 0; k < kXAhead; ++k) {
      const int i = i0 + k * nw, bb = i % B, t = i / B, c = (t * 64 + lane) * 8;
      if (i >= pieces) continue;
      if constexpr (decltype(is_even)::value) xv[k] = load_x8<X>(row_of(bb), c);
      else xv[k] = whole_x8<X>(row_at(bb), c, bb < a.batch ? a.cols : 0);
      if constexpr (X != kQ4F16)  // past the last unit: a group past the row's, or x is zero
        xsc[k] = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(
                       q4_rsrc(a.xscale + (size_t)bb * xgroups, bb < a.batch ? xgroups * 4 : 0),
                       ((t * kStepUnits + (lane >> 2)) >> a.xshift) * 4, 0, 0));
    }
  };
  auto put_ahead = [&](int i0, auto is_even) {
#pragma unroll
    for (int k = 0; k < kXAhead; ++k) {
      const int i = i0 + k * nw, bb = i % B, t = i / B;
      if (i >= pieces) continue;
      if constexpr (!decltype(is_even)::value)
        if (t == a.cols / 512) xv[k] |= cut_x8<X>(row_of(bb), (t * 64 + lane) * 8, a.cols);
      put_x8<B, X, Z>(xs, sums, scaled, xv[k], xsc[k], bb, t, lane);
    }
  };
  int i0 = wv;
  if (even) {
    load_ahead(i0, std::true_type{});
    for (; i0 + kXAhead * nw < pieces; i0 += kXAhead * nw) {
      put_ahead(i0, std::true_type{});
      load_ahead(i0 + kXAhead * nw, std::true_type{});
    }
  } else {  // all of x here, nothing left for later
    for (; i0 < pieces; i0 += kXAhead * nw) {
      load_ahead(i0, std::false_type{});
      put_ahead(i0, std::false_type{});
    }
  }

  // 2. this wave's steps: whole quads, one in nw of the workgroup's; of the
  //    fewer than nw that remain, the steps [first, last)
  const int stride = a.wgs;
  const bool more = (int)blockIdx.x < a.extra;
  const int whole = more ? a.whole[0] : a.whole[1], rest0 = whole * nw;
  const int per = more ? a.per[0] : a.per[1];
  const int rest_steps = (a.quads + more - rest0) * steps;
  const int first = wv * per < rest_steps ? wv * per : rest_steps;
  const int last = first + per < rest_steps ? first + per : rest_steps;
  const int skip = first / steps;
  const int q2 = (int)blockIdx.x + (rest0 + skip) * stride, t2 = first - skip * steps;
  struct Cursor {
    int quad, t, whole, left;  // whole: whole quads to go, this one included
  };
  Cursor at = {(int)blockIdx.x + wv * stride, 0, whole, whole * steps + last - first};
  if (whole == 0) at.quad = q2, at.t = t2;
  auto advance = [&](Cursor& c, int n) {  // returns whether a quad ended
    c.t += n, c.left -= n;
    if (c.t < steps) return false;
    --c.whole;
    c.quad = c.whole > 0 ? c.quad + nw * stride : c.whole == 0 ? q2 : c.quad + stride;
    c.t = c.whole == 0 ? t2 : 0;
    return true;
  };
  auto steps_in_chunk = [&](const Cursor& c) {
    const int n = steps - c.t < c.left ? steps - c.t : c.left;
    return n < kChunk ? n : kChunk;
  };
  Cursor ld = at;  // where the loads are

  const int ul = lane >> 2, r4 = lane & 3;
  const int row_bytes = nunits * 16;
  int lane_off = r4 * row_bytes + ul * 16;
  // formed here: between the loads, the compiler's 64-bit multiply-add can take
  // a load's result register as its unused half, and wait for it
  asm volatile("" : "+v"(lane_off));
  auto load = [&](Q4Chunk<NS>& c) {
    const int n = steps_in_chunk(ld), lt = ld.t;
    const int row = ld.quad * 4, rows = a.rows - row < 4 ? a.rows - row : 4;
    // the step's offset sits in the base, so that the range check is exact; a
    // row's last step may run into the next row, against zeros of x
    const uint8_t* base = a.codes + (size_t)row * row_bytes + lt * (kStepUnits * 16);
    const uint32_t bytes = rows * row_bytes - lt * (kStepUnits * 16);
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const int t = lt + k * (kChunk / NS);
      const int g = ((t * kStepUnits) >> a.gshift) + ul;
      // a group past the row's end: an offset past every buffer, by the sign
      // bit of the difference (a select becomes a branch around the load)
      const int off =
          ((r4 * groups + g) * 2) | ((groups - 1 - g) & (int)0x80000000);
      const uint32_t n2 = k * (kChunk / NS) < n ? (uint32_t)(rows * groups) * 2 : 0;
      c.s[k] = __builtin_amdgcn_raw_buffer_load_b16(
          q4_rsrc(a.scale + (size_t)row * groups, n2), off, 0, 0);
      if constexpr (Z)
        c.z[k] = __builtin_amdgcn_raw_buffer_load_b16(
            q4_rsrc(a.zero + (size_t)row * groups, n2), off, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);  // the scales first: they are waited for first
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      c.w[i] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(q4_rsrc(base, i < n ? bytes : 0),
                                                         lane_off, i * (kStepUnits * 16), 2));
    advance(ld, n);
  };
  Q4Chunk<NS> ring[RING];
#pragma unroll
  for (int d = 0; d < RING; ++d) load(ring[d]);
  if (even) put_ahead(i0, std::true_type{});
  __syncthreads();

  // 3. the steps
  const uint8_t* xl = xs + (ul * B + (r4 < B ? r4 : 0)) * 16;
  const float* sl = sums + ul * B;
  const float* tl = scaled + ul * B;
  // lane of a chunk's scale register that holds this lane's group, step 0, and
  // what a step adds (bytes of a lane index)
  const int from = (((ul >> a.gshift) << 2) | r4) << 2;
  const int from_step = (kStepUnits >> a.gshift) << 4;
  float acc[B];
#pragma unroll
  for (int bb = 0; bb < B; ++bb) acc[bb] = 0.f;

  auto multiply = [&](u32x4_t q, uint32_t sz, int t) {
    const uint8_t* xt = xl + t * x_step_bytes(B, X);
    // e4m3: the codes' unit leaves with the scale (fp16 x: at the store), so that a
    // small scale of x does not push the sum below fp32's normal numbers
    const float s = f16_to_f32(sz) * (X == kQ4E4M3 ? 1.f / code_unit(X) : 1.f);
    const float z = f16_to_f32(sz >> 16);
    const float* sx = sl + t * (kStepUnits * B);
    const float* tx = tl + t * (kStepUnits * B);
    float v[B];
    if constexpr (X == kQ4I8) {
      int4_t c;
#pragma unroll
      for (int bb = 0; bb < B; ++bb) c[bb] = Z ? 0 : __builtin_bit_cast(int, sx[bb]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4_t x = *(const u32x4_t*)(xt + h * slab_bytes(B));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t w = q[2 * h + k];
          c = __builtin_amdgcn_mfma_i32_4x4x4i8((int)x[2 * k], (int)(w & 0x0F0F0F0Fu), c, 0, 0, 0);
          c = __builtin_amdgcn_mfma_i32_4x4x4i8((int)x[2 * k + 1], (int)((w >> 4) & 0x0F0F0F0Fu), c,
                                                0, 0, 0);
        }
      }
#pragma unroll
      for (int bb = 0; bb < B; ++bb) v[bb] = Z ? __builtin_fmaf(z, sx[bb], (float)c[bb]) : (float)c[bb];
    } else {
      // one chain of sums, from -z sum x
      float4_t c;
#pragma unroll
      for (int bb = 0; bb < B; ++bb) c[bb] = Z ? z * sx[bb] : sx[bb];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u32x4_t x = *(const u32x4_t*)(xt + k * slab_bytes(B));
        const uint32_t w = q[k];
        constexpr int b = code_bit(X);
        constexpr uint32_t m = 0x000F000Fu << b;
        c = __builtin_amdgcn_mfma_f32_4x4x4f16(
            __builtin_bit_cast(half4_t, u32x2_t{x.x, x.y}),
            __builtin_bit_cast(half4_t, u32x2_t{(w << b) & m, (w >> (8 - b)) & m}), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_4x4x4f16(
            __builtin_bit_cast(half4_t, u32x2_t{x.z, x.w}),
            __builtin_bit_cast(half4_t, u32x2_t{(w << (b - 4)) & m, (w >> (12 - b)) & m}), c, 0, 0,
            0);
      }
#pragma unroll
      for (int bb = 0; bb < B; ++bb) v[bb] = c[bb];
    }
#pragma unroll
    for (int bb = 0; bb < B; ++bb) {
      // the scale of x last: s times it may be below the normal numbers
      if constexpr (X == kQ4F16) acc[bb] = __builtin_fmaf(s, v[bb], acc[bb]);
      else acc[bb] = __builtin_fmaf(s * v[bb], tx[bb], acc[bb]);
    }
  };
  // lane 4 bb + i < 4 B: the sum of row i of the quad, batch row bb
  auto total = [&]() {
    float r = 0.f;
#pragma unroll
    for (int bb = 0; bb < B; ++bb) {
      const float t = sum_blocks(acc[bb]);
      r = ul == bb ? t : r;
      acc[bb] = 0.f;
    }
    return r;
  };
  auto store = [&](int quad, float r) {
    const int row = quad * 4 + r4;
    if (ul < a.batch && row < a.rows)
      a.y[(size_t)ul * a.rows + row] = X == kQ4F16 ? r * (1.f / code_unit(X)) : r;
  };

  float own = 0.f;  // of a quad that starts in this wave and ends in a later one
  int own_quad = -1;
  auto consume = [&](const Q4Chunk<NS>& c) {
    const int n = steps_in_chunk(at);
    auto step = [&](int i) {
      constexpr int SPL = kChunk / NS;
      // through an empty statement: widened where it was loaded, the wait for
      // the load would be there too
      uint16_t scale = c.s[i / SPL], zero = 0x4800;  // 8.0
      asm volatile("" : "+v"(scale));
      if constexpr (Z) {
        zero = c.z[i / SPL];
        asm volatile("" : "+v"(zero));
      }
      uint32_t sz = (uint32_t)scale | (uint32_t)zero << 16;
      if constexpr (NS < kChunk)
        sz = (uint32_t)__builtin_amdgcn_ds_bpermute(from + (i % SPL) * from_step, (int)sz);
      multiply(c.w[i], sz, at.t + i);
    };
    if (n == kChunk) {  // one block of code: the reads of a step overlap the step before
#pragma unroll
      for (int i = 0; i < kChunk; ++i) step(i);
    } else {
#pragma unroll
      for (int i = 0; i < kChunk - 1; ++i)
        if (i < n) step(i);
    }
    const int quad = at.quad;
    // a piece that continues an earlier wave's: the first of the divided quads
    const bool head = at.whole <= 0 && quad == q2 && t2 != 0;
    const bool ended = advance(at, n);
    if (ended || at.left == 0) {
      const float r = total();
      if (head) {
        if (lane < 4 * B) join[wv * (4 * B) + lane] = r;
      } else if (ended) {
        store(quad, r);
      } else {
        own = r, own_quad = quad;
      }
    }
  };
  if constexpr (RING == 1) {
    if (at.left > 0) consume(ring[0]);
  } else {
    // the loads of the loop are one sequence without branches, so that each
    // wait counts exactly the loads behind the one it is for
    while (ld.left > 0) {  // both chunks hold steps, and a load follows each
      consume(ring[0]);
      load(ring[0]);
      consume(ring[1]);
      load(ring[1]);
    }
    if (at.left > 0) consume(ring[0]);
    if (at.left > 0) consume(ring[1]);
  }
  if (per % steps) {  // the same in every wave: some quad lies in several
    __syncthreads();
    if (own_quad >= 0) {
      const int end = (last + steps - 1) / steps * steps;  // of the quad, among the divided steps
      for (int v = wv + 1; v * per < end && v * per < rest_steps; ++v)
        if (lane < 4 * B) own += join[v * (4 * B) + lane];
      store(own_quad, own);
    }
  }
}

// How the quads of a workgroup are dealt to nw waves, and the chunks that the wave
// with most requests (an even number where it goes round its ring of two).
struct Q4Deal {
  int whole, per, chunks;
};
inline __attribute__((always_inline)) Q4Deal q4_deal(int quads, int steps, int nw) {
  Q4Deal d;
  d.whole = quads / nw;
  const int rest = (quads - d.whole * nw) * steps;
  d.per = (rest + nw - 1) / nw;
  d.chunks = d.whole * ((steps + kChunk - 1) / kChunk);
  // a part that crosses a quad's end may take a chunk more
  if (d.per) d.chunks += (d.per + kChunk - 1) / kChunk + (rest > steps && steps % d.per != 0);
  if (d.chunks > 1) d.chunks += d.chunks & 1;
  return d;
}

template <int B, int X, int NS, bool Z>
int launch_q4_ring(const Q4Call& c, hipStream_t st) {
  const int steps = steps_of(c.cols);
  const size_t lds = q4_lds_bytes(B, X, steps);
  // One workgroup per CU, the quads dealt evenly.  Waves: what costs a CU least,
  // a chunk being about 80 cycles of its load unit (five loads of 16, whether or
  // not a load cut off returns anything) and 1200 cycles of one wave's time, which
  // other waves overlap: 4096x12288 takes 12 waves of two full chunks instead of
  // 16 of four steps and two (batch 4: 9.8 us against 10.7), 4096x4096 takes 8 of
  // one instead of 16 of half a chunk (4.2 us against 4.6).  And enough to bring
  // in the x of four batch rows, whatever the batch: the waves decide where a
  // row's steps are divided, and a row's bits are the same in every batch.  (With
  // the lower bound of batch 1 for all, 1024x12288 batch 4 takes 7.1 us instead
  // of 6.5; with this one, 1024x16384 batch 1 takes 4.9 instead of 4.6.)
  const int cus = device_cus();
  const int quads = (int)(((long long)c.rows + 3) / 4);
  Q4Args a;
  a.codes = c.codes, a.scale = c.scale, a.zero = c.zero;
  a.x = c.x, a.xscale = c.xscale, a.y = c.y;
  a.rows = c.rows, a.cols = c.cols, a.nunits = units_of(c.cols), a.steps = steps;
  a.groups = groups_of(a.nunits, c.gshift), a.gshift = (uint8_t)c.gshift;
  a.xshift = (uint8_t)c.xshift, a.batch = (uint16_t)c.batch;
  a.wgs = quads < cus ? quads : cus;
  a.quads = quads / a.wgs, a.extra = quads % a.wgs;
  const int most = a.quads + (a.extra != 0);
  const int least = (LVQ_MAX_BATCH * steps + 2 * kXAhead - 1) / (2 * kXAhead);
  int nw = kQ4Waves;
  long long best = -1;
  auto consider = [&](auto waves) {  // a constant, so that its divisions are none
    constexpr int n = decltype(waves)::value;
    if (n < kQ4Waves && n < least) return;
    const long long cost = (long long)q4_deal(most, steps, n).chunks * (80 * n + 1200);
    if (best < 0 || cost < best) best = cost, nw = n;
  };
  consider(std::integral_constant<int, 16>{});
  if (most < 8 * kQ4Waves) {  // with more, 16 waves lose little to the last round
    consider(std::integral_constant<int, 14>{});
    consider(std::integral_constant<int, 12>{});
    consider(std::integral_constant<int, 10>{});
    consider(std::integral_constant<int, 8>{});
    consider(std::integral_constant<int, 6>{});
    consider(std::integral_constant<int, 4>{});
    consider(std::integral_constant<int, 3>{});
    consider(std::integral_constant<int, 2>{});
    consider(std::integral_constant<int, 1>{});
  }
  const Q4Deal more = q4_deal(a.quads + 1, steps, nw), fewer = q4_deal(a.quads, steps, nw);
  a.waves = nw;
  a.whole[0] = more.whole, a.whole[1] = fewer.whole;
  a.per[0] = (uint16_t)more.per, a.per[1] = (uint16_t)fewer.per;
  const bool one_chunk = fewer.chunks == 1 && (a.extra == 0 || more.chunks == 1);
  const dim3 grid(a.wgs), block(kWave * nw);
  clear_hip_error();
  if (one_chunk) hipLaunchKernelGGL((q4_gemv_kernel<B, X, NS, Z, 1>), grid, block, lds, st, a);
  else hipLaunchKernelGGL((q4_gemv_kernel<B, X, NS, Z, 2>), grid, block, lds, st, a);
  return launch_status();
}

template <int B, int X, bool Z>
int launch_q4_groups(const Q4Call& c, hipStream_t st) {
  return c.gshift == 0   ? launch_q4_ring<B, X, 4, Z>(c, st)
         : c.gshift == 1 ? launch_q4_ring<B, X, 2, Z>(c, st)
                         : launch_q4_ring<B, X, 1, Z>(c, st);
}

template <int B, int X>
int launch_q4_batch(const Q4Call& c, hipStream_t st) {
  return c.zero ? launch_q4_groups<B, X, true>(c, st) : launch_q4_groups<B, X, false>(c, st);
}

// Three batch rows run as four (the fourth zeros) where their x fits in LDS (up to
// 18,432 columns, 17,408 of e4m3, any of int8), else as two and one, which reads the
// weights twice: 4096x21840 24.6 us, of which the two rows take 13.1 and the one 11.9
// (4096x16384 batch 3 11.9).  Every other x of batch * cols <= 65536 fits.
template <int X>
int launch_q4(Q4Call c, hipStream_t st) {
  const size_t most = device_lds_bytes();
  const int steps = steps_of(c.cols);
  if (c.batch == 3 && q4_lds_bytes(4, X, steps) > most) {
    c.batch = 2;
    const int e = launch_q4<X>(c, st);
    if (e) return e;
    c.batch = 1;
    c.x = (const uint8_t*)c.x + (size_t)2 * c.cols * (X == kQ4F16 ? 2 : 1);
    if (X != kQ4F16) c.xscale += (size_t)2 * groups_of(units_of(c.cols), c.xshift);
    c.y += (size_t)2 * c.rows;
    return launch_q4<X>(c, st);
  }
  const int B = c.batch == 3 ? 4 : c.batch;
  if (q4_lds_bytes(B, X, steps) > most) return LVQ_E_SHAPE;
  return B == 1   ? launch_q4_batch<1, X>(c, st)
         : B == 2 ? launch_q4_batch<2, X>(c, st)
                  : launch_q4_batch<4, X>(c, st);
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
  if (rows && (!y || (cols && (!codes || !scale || !x || (xkind != kQ4F16 && !x_scale)))))
    return LVQ_E_NULL;
  if (!aligned16(codes) || !aligned16(scale) || !aligned16(zero) || !aligned16(x) ||
      !aligned16(x_scale) || !aligned16(y))
    return LVQ_E_ALIGN;
  if ((long long)batch * cols > 65536) return LVQ_E_SHAPE;
  if (rows == 0) return LVQ_OK;
  const size_t ybytes = (size_t)batch * rows * 4;
  const size_t meta = (size_t)rows * group_count(cols, group) * 2;
  if (ranges_overlap(y, ybytes, x, (size_t)batch * cols * (xkind == kQ4F16 ? 2 : 1)) ||
      ranges_overlap(y, ybytes, x_scale, (size_t)batch * group_count(cols, x_group) * 4) ||
      ranges_overlap(y, ybytes, codes, (size_t)rows * ((cols + 31) / 32) * 16) ||
      ranges_overlap(y, ybytes, scale, meta) || ranges_overlap(y, ybytes, zero, meta))
    return LVQ_E_SHAPE;
  if (cols == 0) return zero_output(y, (size_t)batch * rows, st);
  const Q4Call c = {codes, scale, zero, gs, rows, cols, x, x_scale, xs, y, batch};
  if (xkind == kQ4F16) return launch_q4<kQ4F16>(c, st);
  if (xkind == kQ4I8) return launch_q4<kQ4I8>(c, st);
  return launch_q4<kQ4E4M3>(c, st);
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
