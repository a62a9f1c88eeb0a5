// Attention of a few query tokens per sequence over the 4-bit key/value cache.
//
//   o_r = sum_t p_rt v_t / sum_t p_rt,  p_rt = 2^(x_rt - m_r),  x_rt = log2(e) scale q_r k_t
//
// over the tokens t that row r (a query token and one of its heads) sees; m_r is a
// running maximum.  With k_tc = s_tg c_tc + l_tg (c: codes, g: the channel's group)
//
//   q_r k_t       = sum_g s_tg (sum_c q_rc c_tc) + l_tg (sum_c q_rc)
//   sum_t p_rt v_t = sum_t (p_rt s_tg) c_tc + sum_t p_rt l_tg
//
// so both inner sums run on the matrix cores over codes as they are, and scales and low
// ends are applied in fp32: no rounding of a key or a value.  A code inside an fp16's
// mantissa, bits 6..9, is a subnormal, the code times 2^-18; two shifts and masks give
// each pair, and the pages hold the codes in the order in which these pairs are
// operands.  p s is split into two fp16, the rounded value and the rest.
//
// A wave takes 64 tokens at a time, four blocks of 16.  Keys: four products of 16 tokens by
// 16 rows in dim / 32 steps.  Row 4 b + i of product j is token 4 j + i of block b, so that
// lane 16 b + r leaves them with the 16 tokens of block b for row r: exactly the operand
// that the product of the values' channels by rows needs, whose steps run over those tokens.
// Weights never leave their lane.  With 4 or 8 rows the 16 columns repeat them; a
// lane then keeps one or two of its four products' tokens, and its other weights are zeros
// (the columns are summed at the end), so no exponential is computed twice.  Scales
// pass through LDS, to the lanes that need the scales of their tokens.  Workgroups split
// a sequence further, and a second launch joins their parts.
//
// What bounds it, and what it measured (GPU, one call): long sequences, the read of the cache
// with 4 rows or less (64 sequences of 4096 tokens, 8 key/value heads of 128: 57 us, 5.0 TB/s;
// each further token 5.9 TB/s), with 16 rows the vector instructions that unpack the codes and
// make the weights (131072 tokens in groups of 32, 168 MB: 44.6 us in a trace and 4.7 of the join,
// 46 a call). Short ones, the length of the code that a wave runs through once: 1001 tokens of 128
// channels 6.2 us and 3.6 of the join, 490 tokens 7.7 in one launch (6.0 of 64 channels, 11.4 of 256).

#include "kv_cache.h"

namespace lvq {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttWaves = 4;    // of a workgroup, more where that saves time
constexpr int kAttMostWaves = 8;
constexpr int kAttWhole = 8;    // blocks of a sequence that a workgroup takes alone
constexpr int kAttTokens = 64;  // of a wave at a time
constexpr uint32_t kCodeMask = 0x03C003C0u;
constexpr float kCodeUnit = 0x1p18f;

struct AttArgs {
  KvPages c;
  uint16_t heads, queries;
  const int32_t* lens;
  const void* q;
  void* out;
  float* parts;   // [seqs][kv_heads][splits][rows][dim], then {maximum, sum} of each
  int64_t q_stride;  // values
  float scale, scale_rest;  // of the logits, in powers of two: rounded down, and the rest
  int window, splits;
  uint16_t tiles;  // of rows
  uint8_t q_type, out_type, waves;
  uint16_t round;  // sequences that the chip begins at a time; 0: taken as they come
};
static_assert(sizeof(AttArgs) < 128, "launches of 128 bytes and more are slower");

// The tokens any query of a sequence sees, in blocks of 64, and over how many workgroups
// they are split: block n (from the first) goes to wave n % waves of workgroup n / waves,
// all modulo the whole.  So a workgroup's first blocks do not depend on the length, and
// their pages' numbers are asked for before it is known.
struct Span {
  int first, last, parts, len;
};
__device__ __forceinline__ Span att_span(const KvPages& c, int len, int queries, int window,
                                         int splits, int waves) {
  Span s;
  const int most = c.pages ? c.max_pages << c.page_shift : 0;
  s.len = len < 0 ? 0 : len > most ? most : len;
  int first = 0;
  if (window > 0) {
    first = s.len - queries - window + 1;  // of the first query's window
    first = first < 0 ? 0 : first / kAttTokens;
  }
  s.first = first;
  s.last = (s.len + kAttTokens - 1) / kAttTokens;
  const int parts = (s.last - s.first + waves - 1) / waves;
  s.parts = parts < 1 ? 1 : parts < splits ? parts : splits;
  return s;
}

// The sequence of place z in the order of work: by length, the longest first, every other
// round backwards, so that a CU that began with a long one goes on with a short one (64
// sequences of up to 8192 tokens take 71 us so, 84 as they come). Up to 64 sequences.
__device__ __forceinline__ int att_in_order(const AttArgs& a, int z, int lane) {
  const int mine = lane < a.c.seqs ? a.lens[lane] : 0;
  int rank = lane < a.c.seqs ? 0 : kWave;
  for (int j = 0; j < a.c.seqs; ++j) {
    const int other = __builtin_amdgcn_readlane(mine, j);
    rank += other > mine || (other == mine && j < lane);
  }
  const int turn = z / a.round, end = (turn + 1) * a.round;
  const int want = turn & 1 ? (end < a.c.seqs ? end : a.c.seqs) - 1 - (z - turn * a.round) : z;
  return __builtin_ctzll(__ballot(rank == want));
}

__device__ __forceinline__ float att_f16(uint32_t b) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

template <int CTRL>
__device__ __forceinline__ float dpp_max_f(float v) {
  const int i = __builtin_bit_cast(int, v);
  return fmaxf(v, __builtin_bit_cast(
                      float, __builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, false)));
}

// Over the lanes of one row: the 16 / RT of a quarter that share it, and the quarters.
template <int RT>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (RT <= 8) v = dpp_max_f<0x128>(v);  // row_ror:8
  if constexpr (RT <= 4) v = dpp_max_f<0x124>(v);  // row_ror:4
  if constexpr (RT <= 1) {
    v = dpp_max_f<0x4E>(v);
    v = dpp_max_f<0xB1>(v);
  }
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
  u = __builtin_bit_cast(uint32_t, v);
  auto q = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)q[0]),
               __builtin_bit_cast(float, (uint32_t)q[1]));
}
// Over the columns of a row, then (row_sum) the quarters; every step adds the same two
// values on both sides.
template <int RT>
__device__ __forceinline__ float column_sum(float v) {
  if constexpr (RT <= 8) v = dpp_add<0x128, 0xF>(v);
  if constexpr (RT <= 4) v = dpp_add<0x124, 0xF>(v);
  return v;
}
__device__ __forceinline__ float quarter_sum(float v) {
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
  u = __builtin_bit_cast(uint32_t, v);
  auto q = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)q[0]) + __builtin_bit_cast(float, (uint32_t)q[1]);
}

// Orders a wave's LDS accesses (its LDS instructions execute in order).
__device__ __forceinline__ void lds_order() {
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ half8_t codes8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(half8_t, u32x4{a & kCodeMask, b & kCodeMask, c & kCodeMask,
                                           d & kCodeMask});
}

__device__ __forceinline__ void att_store4(void* out, int type, size_t at, f32x4_t v) {
  if (type == LVQ_F32) {
    __builtin_memcpy((float*)out + at, &v, 16);
    return;
  }
  uint32_t b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (type == LVQ_F16)
      b[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i + 1]) << 16;
    else
      b[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i + 1]) << 16;
  }
  __builtin_memcpy((uint16_t*)out + at, b, 8);
}

// LDS of a wave: the scales and low ends of 64 tokens; then, in the same place, its part of
// the result [RT][DIM], maxima, sums and low ends.
constexpr int att_part_bytes(int RT, int dim) { return RT * dim * 4; }
constexpr int att_wave_bytes(int RT, int dim, int groups) {
  const int a = 2 * groups * kAttTokens * 4;
  const int b = att_part_bytes(RT, dim) + (2 + groups) * RT * 4;
  return a > b ? a : b;
}

// Waves of a SIMD that the registers are to leave room for.
constexpr int att_waves(int dim, int groups) {
  return dim == 64 || (dim == 128 && groups == 1) ? 3 : 2;
}

template <int DIM, int RT, int NG>
__global__ void __launch_bounds__(kAttMostWaves* kWave, att_waves(DIM, NG))
    attend_kernel(AttArgs a) {
  constexpr int KS = DIM / 32;       // steps of 32 channels
  constexpr int GS = KS / NG;        // of a group
  constexpr int NT = RT / 4;         // products (of four tokens a lane) that a lane keeps
  constexpr int kLds = att_wave_bytes(RT, DIM, NG), kPart = att_part_bytes(RT, DIM);
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int nw = a.waves;
  const int lane = threadIdx.x & (kWave - 1), t16 = lane & 15, quarter = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int seq = a.round ? att_in_order(a, blockIdx.z, lane) : blockIdx.z, part = blockIdx.y;
  const int head = blockIdx.x / a.tiles, tile = blockIdx.x - head * a.tiles;
  const int per = a.heads / a.c.kv_heads, rows = per * a.queries;
  const int row0 = tile * 16;
  const int stride = nw * a.splits;
  const int len = a.lens[seq];
  int b = part * nw + wv;
  if (a.window > 0) b += att_span(a.c, len, a.queries, a.window, a.splits, a.waves).first;

  uint8_t* const lds = smem + wv * kLds;
  const int64_t page_size = kv_page_size(a.c);
  constexpr int kBlock = kv_block_bytes(DIM, NG);
  const int blocks_mask = (1 << (a.c.page_shift - 4)) - 1;
  const int32_t* table = a.c.table + (int64_t)seq * a.c.max_pages;
  const uint8_t* pool = a.c.pool + (int64_t)head * (blocks_mask + 1) * kBlock;

  // the page of block `blk` of 64 tokens, and where the block lies (a page outside the
  // pool: the first page, read and not used)
  auto page_of = [&](int b, int blk) {
    const int at = (b * kAttTokens + 16 * blk) >> a.c.page_shift;
    return table[at < a.c.max_pages ? at : a.c.max_pages - 1];
  };
  auto outside = [&](int page) { return page < 0 || page >= a.c.pages; };
  auto block_at = [&](int b, int blk, int page) {
    return pool + (outside(page) ? 0 : page) * page_size +
           ((4 * b + blk) & blocks_mask) * (int64_t)kBlock;
  };
  // a lane reads the keys of block t16 / 4, tokens 4 j + t16 % 4, and the values and
  // the scales of block `quarter`
  const int kblk = t16 >> 2;
  struct Tokens {
    uint32_t k[4][KS];
    u32x4 v[KS];
    uint32_t ks[NG], vs[NG];
  };
  Tokens x;
  auto load_k = [&](const uint8_t* key, const uint8_t* own) {
    const uint8_t* p = key + (t16 & 3) * (DIM / 2) + quarter * (DIM / 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) __builtin_memcpy(x.k[j], p + j * 2 * DIM, KS * 4);
#pragma unroll
    for (int g = 0; g < NG; ++g) x.ks[g] = *(const uint32_t*)(own + 16 * DIM + 64 * g + 4 * t16);
#pragma unroll
    for (int g = 0; g < NG; ++g)
      x.vs[g] = *(const uint32_t*)(own + 16 * DIM + 64 * (NG + g) + 4 * t16);
  };
  auto load_v = [&](const uint8_t* own) {
#pragma unroll
    for (int s = 0; s < KS; ++s) __builtin_memcpy(&x.v[s], own + 8 * DIM + (16 * s + t16) * 16, 16);
  };

  // the pages' numbers of this wave's first two blocks, then the length
  int bn = b + stride, key_page = -1, page = -1, key_page_n = -1, page_n = -1;
  if (a.c.max_pages) {
    key_page = page_of(b, kblk), page = page_of(b, quarter);
    key_page_n = page_of(bn, kblk), page_n = page_of(bn, quarter);
  }
  const Span sp = att_span(a.c, len, a.queries, a.window, a.splits, a.waves);
  if (part >= sp.parts) return;
  const int b1 = sp.last;
  // the loads of the loop are one sequence without branches, so that each wait counts
  // just the loads behind the one it is for: at the end the last block again
  if (bn >= b1) bn = b, key_page_n = key_page, page_n = page;
  if (b < b1) {
    const uint8_t* own = block_at(b, quarter, page);
    load_k(block_at(b, kblk, key_page), own);
    load_v(own);
  }

  // q: operand column t16 (row t16 % RT), channels 32 s + 8 quarter .. + 7 of step s
  half8_t qa[KS];
  float qs[NG], unit = a.scale * kCodeUnit;  // sums of the row's q over a group, a logit's unit
  float unit_rest = a.scale_rest * kCodeUnit;
  const int r = row0 + (t16 & (RT - 1));
  int see_first = 0, see_last = sp.len - 1;  // rows past the last: not stored
  {
    const bool real = r < rows;
    const int query = real ? r / per : 0, h = head * per + (real ? r - query * per : 0);
    if (real) {
      see_last = sp.len - a.queries + query;
      see_first = a.window > 0 ? see_last - a.window + 1 : 0;
    }
    const uint16_t* row = (const uint16_t*)a.q +
                          ((int64_t)seq * a.queries + query) * a.q_stride + (int64_t)h * DIM;
    uint4 raw[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) __builtin_memcpy(&raw[s], row + 32 * s + 8 * quarter, 16);
#pragma unroll
    for (int g = 0; g < NG; ++g) qs[g] = 0.f;
    if (a.q_type == LVQ_F16) {
#pragma unroll
      for (int s = 0; s < KS; ++s) qa[s] = __builtin_bit_cast(half8_t, raw[s]);
    } else {
      // bf16: the row times a power of two that brings its largest value to [1, 2), where
      // fp16 holds the eight bits of every value down to 2^-17 of it
      uint32_t top = 0;
      float v[KS][8];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint32_t w[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t bits = (i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
          v[s][i] = __builtin_bit_cast(float, bits);
          const uint32_t m = bits & 0x7F800000u;
          top = top > m ? top : m;
        }
      }
      uint32_t o = __shfl_xor(top, 16, kWave);
      top = top > o ? top : o;
      o = __shfl_xor(top, 32, kWave);
      top = top > o ? top : o;
      // an infinity or a NaN, or nothing but zeros and subnormal numbers: as it is
      top = top == 0x7F800000u || top == 0 ? 0x3F800000u : top;
      top = top < 0x01000000u ? 0x01000000u : top > 0x7E000000u ? 0x7E000000u : top;
      const float down = __builtin_bit_cast(float, 0x7F000000u - top);
      unit *= __builtin_bit_cast(float, top), unit_rest *= __builtin_bit_cast(float, top);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) qa[s][i] = (_Float16)(v[s][i] * down);
    }
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) qs[s / GS] += (float)qa[s][i];
#pragma unroll
    for (int g = 0; g < NG; ++g) qs[g] = quarter_sum(qs[g]) * (1.f / kCodeUnit);
    // above 0, so that times minus infinity they are no NaN (logits in them are 0 all the same)
    unit = fmaxf(unit, 0x1p-126f), unit_rest = fmaxf(unit_rest, 0x1p-126f);
  }
  // tokens that every row sees, and the first that any does
  int all_first = 0, any_first = 0, all_last;
  {
    const int q0 = row0 / per, q1 = (row0 + RT < rows ? row0 + RT - 1 : rows - 1) / per;
    all_last = sp.len - a.queries + q0;
    if (a.window > 0) {
      all_first = sp.len - a.queries + q1 - a.window + 1;
      any_first = sp.len - a.queries - a.window + 1;
    }
  }
  // the products that a lane keeps: its n-th is number product(n)
  const int col = RT == 4 ? t16 >> 2 : RT == 8 ? t16 >> 3 : 0;
  auto product = [&](int n) { return RT == 4 ? col : RT == 8 ? 2 * n + col : n; };
  uint32_t keep[4];  // operand masks: all ones where the lane keeps product j
#pragma unroll
  for (int j = 0; j < 4; ++j)
    keep[j] = RT == 4 ? (col == j ? ~0u : 0u) : RT == 8 ? (col == (j & 1) ? ~0u : 0u) : ~0u;

  float m = -__builtin_inff(), l = 0.f, low[NG];
  f32x4_t acc[KS][2];
#pragma unroll
  for (int g = 0; g < NG; ++g) low[g] = 0.f;
#pragma unroll
  for (int s = 0; s < KS; ++s) acc[s][0] = acc[s][1] = f32x4_t{0, 0, 0, 0};
  // the weights' unit: 2^6 over a power of two above the largest scale so far
  float smax = 0.f, pu = 1.f;

  for (; b < b1; b += stride) {
    const int t0 = b * kAttTokens;
    const bool bad = outside(page);
    const bool edge = t0 < all_first || t0 + kAttTokens - 1 > all_last || __any(bad);
    // ---- scales into LDS; the largest of the values' (of tokens that some row sees)
    float top = 0.f;
    {
      uint32_t ks[NG], vs[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) ks[g] = x.ks[g], vs[g] = x.vs[g];
      // a scale or low end that is not finite becomes a NaN of the token's logit: zero times it is
      // one, and joins the first pair
      lvq_half2 not_a_number = {0, 0};
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (uint32_t w : {ks[g], vs[g]})
          not_a_number = __builtin_elementwise_fma(as_half2(w), lvq_half2{0, 0}, not_a_number);
      ks[0] = __builtin_bit_cast(uint32_t, as_half2(ks[0]) + not_a_number);
      if (edge) {
        // what no row sees is 0, whatever it holds, and so is a value that is not finite: nothing
        // for the rows that do not see it
        const int tok = t0 + lane;
        const bool none = bad || tok >= sp.len || tok < any_first;
        bool wild = false;
#pragma unroll
        for (int g = 0; g < NG; ++g)
          wild |= (vs[g] & 0x7C00u) == 0x7C00u || (vs[g] & 0x7C000000u) == 0x7C000000u;
        if (none || wild)
#pragma unroll
          for (int g = 0; g < NG; ++g) vs[g] = 0;
      }
      lds_order();
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        *(uint32_t*)(lds + (g * kAttTokens + lane) * 4) = ks[g];
        *(uint32_t*)(lds + ((NG + g) * kAttTokens + lane) * 4) = vs[g];
        const float s = fabsf(att_f16(vs[g]));
        top = s < __builtin_inff() ? fmaxf(top, s) : top;
      }
      lds_order();
    }
    // ---- logits
    float lg[NT][4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4_t d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int s = g * GS; s < (g + 1) * GS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = x.k[j][s];
          d[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes8(w << 6, w << 2, w >> 2, w >> 6),
                                                        qa[s], d[j], 0, 0, 0);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4_t e;
        if constexpr (RT == 4) e = col & 2 ? (col & 1 ? d[3] : d[2]) : (col & 1 ? d[1] : d[0]);
        else if constexpr (RT == 8)  // by value: a choice of whole vectors goes through memory
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = col ? d[2 * n + 1][i] : d[2 * n][i];
        else e = d[n];
        const u32x4 sl =
            *(const u32x4*)(lds + (g * kAttTokens + 16 * quarter + 4 * product(n)) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = __builtin_fmaf(att_f16(sl[i]), e[i], g ? lg[n][i] : 0.f);
          lg[n][i] = __builtin_fmaf(att_f16(sl[i] >> 16), qs[g], c);
        }
      }
      if constexpr (NG > 1) __builtin_amdgcn_sched_barrier(0);
    }
    // ---- the next tokens' keys and scales
    const int page_b = page_n;
    const uint8_t* own_n = block_at(bn, quarter, page_n);
    const uint8_t* key_n = block_at(bn, kblk, key_page_n);
    bn = bn + stride < b1 ? bn + stride : bn;
    key_page_n = page_of(bn, kblk);
    page_n = page_of(bn, quarter);
    load_k(key_n, own_n);
    // ---- what the row does not see
    if (edge) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = t0 + 16 * quarter + 4 * product(n) + i;
          if (bad || tok < see_first || tok > see_last) lg[n][i] = -__builtin_inff();
        }
    }
    // ---- maximum: left behind by up to 2^8, so that it seldom changes
    float big = lg[0][0];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) big = fmaxf(big, lg[n][i]);
    if (__any(top > smax || big * unit > m + 8.f)) {
      const float old_pu = pu;
      smax = row_max<1>(fmaxf(top, smax));
      if (smax > 0.f) {
        const uint32_t e = __builtin_bit_cast(uint32_t, smax) & 0x7F800000u;
        pu = __builtin_bit_cast(float, 0x81800000u - e);
      }
      const float nm = fmaxf(m, row_max<RT>(big) * unit);
      float f = m == nm ? 1.f : __builtin_amdgcn_exp2f(m - nm);  // 0 from minus infinity
      m = nm;
      f *= pu / old_pu;
      l *= f;
#pragma unroll
      for (int g = 0; g < NG; ++g) low[g] *= f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[s][h] *= f;
    }
    // ---- weights
    float p[NT][4];
    const float mi = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the unit's rounding would change logits by 2^-24 of themselves, weights by that times
        // the logit (128 channels, 131072 tokens: 1e-5 of the result); in the weights'
        // unit, a power of two
        const float x = __builtin_fmaf(lg[n][i], unit_rest, __builtin_fmaf(lg[n][i], unit, -mi));
        p[n][i] = __builtin_amdgcn_exp2f(x) * pu;
        l += p[n][i];
      }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // p s, the rounded value and the rest, in the order of the values' pairs: tokens 0 and
      // 2, 1 and 3 of four
      uint32_t hi[NT][2], rest[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const u32x4 sl =
            *(const u32x4*)(lds + ((NG + g) * kAttTokens + 16 * quarter + 4 * product(n)) * 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          lvq_half2 h, t;
          float w[2], s[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            w[i] = p[n][2 * i + k], s[i] = att_f16(sl[2 * i + k]);
            h[i] = (_Float16)(w[i] * s[i]);
            low[g] = __builtin_fmaf(w[i], att_f16(sl[2 * i + k] >> 16), low[g]);
          }
          // the rounded values as they are, for the rests too: rounded anew from w s by an
          // instruction that multiplies and rounds at once, a value between two fp16 may be
          // the other of them
          uint32_t both = __builtin_bit_cast(uint32_t, h);
          asm("" : "+v"(both));
          h = __builtin_bit_cast(lvq_half2, both);
#pragma unroll
          for (int i = 0; i < 2; ++i) t[i] = (_Float16)__builtin_fmaf(w[i], s[i], -(float)h[i]);
          hi[n][k] = both;
          rest[n][k] = __builtin_bit_cast(uint32_t, t);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // products 2 k and 2 k + 1
        const int n0 = RT == 4 ? 0 : RT == 8 ? k : 2 * k, n1 = RT == 16 ? n0 + 1 : n0;
        const uint32_t k0 = keep[2 * k], k1 = keep[2 * k + 1];
        const half8_t w0 = __builtin_bit_cast(
            half8_t, u32x4{hi[n0][0] & k0, hi[n0][1] & k0, hi[n1][0] & k1, hi[n1][1] & k1});
        const half8_t w1 = __builtin_bit_cast(
            half8_t, u32x4{rest[n0][0] & k0, rest[n0][1] & k0, rest[n1][0] & k1, rest[n1][1] & k1});
#pragma unroll
        for (int s = g * GS; s < (g + 1) * GS; ++s) {
          const uint32_t c0 = x.v[s][2 * k], c1 = x.v[s][2 * k + 1];
          const half8_t vl = codes8(c0 << 6, c0 >> 2, c1 << 6, c1 >> 2);
          const half8_t vh = codes8(c0 << 2, c0 >> 6, c1 << 2, c1 >> 6);
          acc[s][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vl, w0, acc[s][0], 0, 0, 0);
          acc[s][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vh, w0, acc[s][1], 0, 0, 0);
          acc[s][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vl, w1, acc[s][0], 0, 0, 0);
          acc[s][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vh, w1, acc[s][1], 0, 0, 0);
        }
      }
      if constexpr (NG > 1) __builtin_amdgcn_sched_barrier(0);
    }
    load_v(own_n);
    page = page_b;
  }

  // ---- this wave's part: maxima, sums and the result by row
  lds_order();
  float* const part_o = (float*)lds;
  float* const part_m = (float*)(lds + att_part_bytes(RT, DIM));
  float* const part_l = part_m + RT;
  const float back = 1.f / pu, sum = quarter_sum(column_sum<RT>(l)) * back;
  if (lane < RT) part_m[lane] = m, part_l[lane] = sum;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float lo = quarter_sum(column_sum<RT>(low[g])) * back;
#pragma unroll
    for (int s = g * GS; s < (g + 1) * GS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4_t v = acc[s][h];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(column_sum<RT>(v[i]), back * kCodeUnit, lo);
        if (t16 < RT) *(f32x4_t*)(part_o + t16 * DIM + 32 * s + 16 * h + 4 * quarter) = v;
      }
  }
  __syncthreads();

  // ---- the workgroup's: four channels of a row per thread
  for (int at4 = threadIdx.x; at4 < RT * (DIM / 4); at4 += nw * kWave) {
    const int r = at4 / (DIM / 4), c = (at4 - r * (DIM / 4)) * 4;
    if (row0 + r >= rows) break;
    float most = -__builtin_inff(), sum = 0.f;
    f32x4_t v = {0, 0, 0, 0};
    // four waves at a time, all their values asked for at once
    for (int w0 = 0; w0 < nw; w0 += kAttWaves) {
      float mw[kAttWaves], lw[kAttWaves];
      f32x4_t ow[kAttWaves];
#pragma unroll
      for (int w = 0; w < kAttWaves; ++w) {
        const uint8_t* from = smem + (w0 + w) * kLds;
        mw[w] = ((const float*)(from + kPart))[r];
        lw[w] = ((const float*)(from + kPart))[RT + r];
        ow[w] = *(const f32x4_t*)((const float*)from + r * DIM + c);
      }
      float top = most;
#pragma unroll
      for (int w = 0; w < kAttWaves; ++w) top = fmaxf(top, mw[w]);
      const float f = most == top ? 1.f : __builtin_amdgcn_exp2f(most - top);
      most = top, sum *= f, v *= f;
#pragma unroll
      for (int w = 0; w < kAttWaves; ++w) {
        const float e = mw[w] == top ? 1.f : __builtin_amdgcn_exp2f(mw[w] - top);
        sum = __builtin_fmaf(lw[w], e, sum);
        v += ow[w] * e;
      }
    }
    if (sp.parts == 1) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int query = (row0 + r) / per, h = head * per + (row0 + r) - query * per;
      att_store4(a.out, a.out_type,
                 (((size_t)seq * a.queries + query) * a.heads + h) * DIM + c, v * inv);
    } else {
      const size_t n = (size_t)rows * a.splits;
      const size_t at = ((size_t)seq * a.c.kv_heads + head) * n + (size_t)part * rows + row0 + r;
      __builtin_memcpy(a.parts + at * DIM + c, &v, 16);
      if (c == 0) {
        float* ml = a.parts + (size_t)a.c.seqs * a.c.kv_heads * n * DIM + 2 * at;
        ml[0] = most, ml[1] = sum;
      }
    }
  }
}

// Joins the parts of a row: a workgroup per row, its parts dealt to groups of DIM / 4
// threads, four channels per thread.  The parts are asked for before the length says how many
// there are (the others hold anything, within the workspace), so that it all takes one trip.
template <int DIM>
__global__ void __launch_bounds__(256) attend_join_kernel(AttArgs a) {
  constexpr int T = DIM / 4, N = 256 / T, U = 8;
  __shared__ f32x4_t part[N][T];
  __shared__ float maxima[N], sums[N];
  const int per = a.heads / a.c.kv_heads, rows = per * a.queries;
  const int seq = blockIdx.y, head = blockIdx.x / rows, r = blockIdx.x - head * rows;
  const int len = a.lens[seq];
  const size_t n = (size_t)rows * a.splits;
  const size_t at = ((size_t)seq * a.c.kv_heads + head) * n + r;
  const float* ml = a.parts + (size_t)a.c.seqs * a.c.kv_heads * n * DIM + 2 * at;
  const float* o = a.parts + at * DIM;
  const int g = threadIdx.x / T, c = threadIdx.x - g * T;
  float big = -__builtin_inff(), sum = 0.f;
  f32x4_t v = {0, 0, 0, 0};
  int parts = a.splits;
  for (int p0 = g; p0 < parts; p0 += U * N) {
    f32x4_t w[U];
    float mp[U], lp[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int p = p0 + k * N < a.splits ? p0 + k * N : p0;
      __builtin_memcpy(&w[k], o + (size_t)p * rows * DIM + 4 * c, 16);
      mp[k] = ml[(size_t)2 * p * rows], lp[k] = ml[(size_t)2 * p * rows + 1];
    }
    parts = att_span(a.c, len, a.queries, a.window, a.splits, a.waves).parts;
    float top = big;
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (p0 + k * N < parts) top = fmaxf(top, mp[k]);
    const float f = big == top ? 1.f : __builtin_amdgcn_exp2f(big - top);
    big = top, sum *= f, v *= f;
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (p0 + k * N < parts) {
        const float e = mp[k] == top ? 1.f : __builtin_amdgcn_exp2f(mp[k] - top);
        sum = __builtin_fmaf(lp[k], e, sum);
        v += w[k] * e;
      }
  }
  parts = att_span(a.c, len, a.queries, a.window, a.splits, a.waves).parts;
  if (parts == 1) return;  // written by its only workgroup
  part[g][c] = v;
  if (c == 0) maxima[g] = big, sums[g] = sum;
  __syncthreads();
  if (g == 0) {
    float top = big;
    for (int k = 1; k < N; ++k) top = fmaxf(top, maxima[k]);
    sum = 0.f, v = f32x4_t{0, 0, 0, 0};
    for (int k = 0; k < N; ++k) {
      const float e = maxima[k] == top ? 1.f : __builtin_amdgcn_exp2f(maxima[k] - top);
      sum = __builtin_fmaf(sums[k], e, sum);
      v += part[k][c] * e;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int query = r / per, h = head * per + r - query * per;
    att_store4(a.out, a.out_type,
               (((size_t)seq * a.queries + query) * a.heads + h) * DIM + 4 * c, v * inv);
  }
}

// ---------------------------------------------------------------- launch

// Blocks of 64 tokens that a sequence has at most (that its queries see).
inline long long att_blocks(const KvPages& c, int queries, int window) {
  long long tokens = (long long)c.max_pages << c.page_shift;
  if (window > 0 && (long long)window + queries + kAttTokens < tokens)
    tokens = (long long)window + queries + kAttTokens;
  return (tokens + kAttTokens - 1) / kAttTokens;
}

// How a sequence's tokens are split: waves of a workgroup and, at most, workgroups.
struct Split {
  int waves, parts;
};
inline Split att_split(const KvPages& c, int queries, int window, int tiles) {
  const long long n = att_blocks(c, queries, window), wgs = (long long)c.seqs * c.kv_heads * tiles;
  const int cus = device_cus();
  // Few tokens: a workgroup alone, without the second launch, and of eight waves if it has a CU
  // to itself (500 tokens of 128 channels, 8 key/value heads: 16 sequences 8.0 us; 57
  // sequences 11.5 us with four waves, 14.4 with eight, of which a CU then holds one)
  if (n <= kAttWhole) return {n > kAttWaves && wgs < cus ? kAttMostWaves : kAttWaves, 1};
  // Else enough workgroups to fill the chip once, two per CU. A few too many would begin when the
  // first have ended, so parts are rounded down (7 of 60000 tokens: 73 parts 15.2 us, 74 18.0;
  // 72 of up to 3733: 7 parts 12.2, 8 13.6), but for less than four, where a third fewer cost
  // more (160 of up to 6000: 3 parts 21.4, 4 19.2).
  const long long down = 2LL * cus / (wgs > 0 ? wgs : 1);
  const long long want = down < 4 ? (2LL * cus + wgs - 1) / (wgs > 0 ? wgs : 1) : down;
  // and no more than there are tokens for
  const long long most = (n + kAttWaves - 1) / kAttWaves, parts = want < most ? want : most;
  return {kAttWaves, parts < 1 ? 1 : (int)parts};
}

inline size_t att_space(const KvPages& c, int heads, int queries, int splits) {
  return splits == 1 ? 0 : (size_t)c.seqs * heads * queries * splits * (c.dim + 2) * 4;
}

template <int DIM, int RT, int NG>
int launch_attend(const AttArgs& a, hipStream_t st) {
  const dim3 grid(a.c.kv_heads * a.tiles, a.splits, a.c.seqs), block(a.waves * kWave);
  clear_hip_error();
  hipLaunchKernelGGL((attend_kernel<DIM, RT, NG>), grid, block,
                     a.waves * att_wave_bytes(RT, DIM, NG), st, a);
  if (a.splits > 1)
    hipLaunchKernelGGL(attend_join_kernel<DIM>, dim3(a.heads * a.queries, a.c.seqs), dim3(256), 0,
                       st, a);
  return launch_status();
}

template <int DIM, int NG>
int launch_rows(const AttArgs& a, int rows, hipStream_t st) {
  return rows <= 4   ? launch_attend<DIM, 4, NG>(a, st)
         : rows <= 8 ? launch_attend<DIM, 8, NG>(a, st)
                     : launch_attend<DIM, 16, NG>(a, st);
}

template <int DIM>
int launch_groups(const AttArgs& a, int rows, hipStream_t st) {
  if (a.c.groups == 1) return launch_rows<DIM, 1>(a, rows, st);
  if (a.c.groups == 2) return launch_rows<DIM, 2>(a, rows, st);
  if constexpr (DIM >= 128)
    if (a.c.groups == 4) return launch_rows<DIM, 4>(a, rows, st);
  if constexpr (DIM >= 256)
    if (a.c.groups == 8) return launch_rows<DIM, 8>(a, rows, st);
  return LVQ_E_SHAPE;
}

// What lvq_attend and its workspace's size check of the sizes.
inline int att_sizes(const KvPages& c, int heads, int queries) {
  if (heads < 1 || heads > kKvMaxHeads || heads % c.kv_heads || queries < 1 ||
      queries > LVQ_MAX_QUERIES || c.seqs > 65535)
    return LVQ_E_SHAPE;
  return LVQ_OK;
}

inline int att_tiles(const KvPages& c, int heads, int queries) {
  return (heads / c.kv_heads * queries + 15) / 16;
}

}  // namespace lvq

using namespace lvq;

extern "C" size_t lvq_attend_workspace(const lvq_kv_cache* cache, int heads, int queries) {
  KvPages c;
  if (kv_pages(cache, &c) || att_sizes(c, heads, queries)) return 0;
  return att_space(c, heads, queries,
                   att_split(c, queries, 0, att_tiles(c, heads, queries)).parts);
}

extern "C" int lvq_attend(const lvq_kv_cache* cache, const void* q, int q_type, int64_t q_stride,
                          int heads, int queries, const int32_t* lens, float scale, int window,
                          void* out, int out_type, void* workspace, size_t workspace_bytes,
                          void* stream) {
  AttArgs a;
  int e = kv_pages(cache, &a.c);
  if (e) return e;
  e = att_sizes(a.c, heads, queries);
  if (e) return e;
  if ((q_type != LVQ_F16 && q_type != LVQ_BF16) ||
      (out_type != LVQ_F32 && out_type != LVQ_F16 && out_type != LVQ_BF16) || window < 0 ||
      !(scale > 0.f && scale < __builtin_inff()))
    return LVQ_E_SHAPE;
  const int64_t cols = (int64_t)heads * a.c.dim, n = (int64_t)a.c.seqs * queries;
  if (q_stride < cols || q_stride > (INT64_MAX >> 4) / (n > 0 ? n : 1)) return LVQ_E_SHAPE;
  if (a.c.seqs == 0) return LVQ_OK;
  if (!q || !lens || !out) return LVQ_E_NULL;
  if ((uintptr_t)q % 2 || (uintptr_t)lens % 4 || !aligned16(out) || !aligned16(workspace))
    return LVQ_E_ALIGN;
  const int rows = heads / a.c.kv_heads * queries;
  a.tiles = (uint16_t)att_tiles(a.c, heads, queries);
  const Split split = att_split(a.c, queries, window, a.tiles);
  a.splits = split.parts, a.waves = (uint8_t)split.waves;
  // in order where a workgroup may have long to run, 32 blocks or more: it costs a trip to memory (as
  // they come and in order, sequences of up to so many tokens, 8 heads of 128.  64, one part each:
  // 1024 14.9, 15.8 us; 2048 22.7, 20.9; 8192 69, 56.  Below 32 blocks mixed: 16, four parts, 4096
  // 17.9, 16.9; 64 of 2 heads, four parts, 2048 13.3, 16.4, 8192 26.1, 24.4)
  const int per_seq = a.c.kv_heads * a.tiles * a.splits;
  const bool ordered = a.c.seqs > 1 && a.c.seqs <= kWave &&
                       att_blocks(a.c, queries, window) >= 32LL * a.splits;
  a.round = (uint16_t)(!ordered ? 0 : per_seq < device_cus() ? device_cus() / per_seq : 1);
  const size_t space = att_space(a.c, heads, queries, a.splits);
  if (space && !workspace) return LVQ_E_NULL;
  if (workspace_bytes < space) return LVQ_E_SHAPE;
  const size_t made_bytes[2] = {(size_t)n * cols * (out_type == LVQ_F32 ? 4 : 2), space};
  const void* made[2] = {out, workspace};
  const void* in[4] = {q, lens, a.c.pool, a.c.table};
  const size_t in_bytes[4] = {((size_t)(n - 1) * q_stride + cols) * 2, (size_t)a.c.seqs * 4,
                              kv_pool_bytes(a.c), kv_table_bytes(a.c)};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 4; ++j)
      if (ranges_overlap(made[i], made_bytes[i], in[j], in_bytes[j])) return LVQ_E_SHAPE;
  if (ranges_overlap(made[0], made_bytes[0], made[1], made_bytes[1])) return LVQ_E_SHAPE;
  a.lens = lens, a.q = q, a.out = out, a.parts = (float*)workspace, a.q_stride = q_stride;
  // a window past any length is none that matters, and keeps sums of positions in range
  const double powers = (double)scale * 1.4426950408889634;
  a.scale = (float)powers;
  if ((double)a.scale > powers) a.scale = __builtin_nextafterf(a.scale, 0.f);
  a.scale_rest = (float)(powers - (double)a.scale), a.window = window < (1 << 30) ? window : 1 << 30;
  a.heads = (uint16_t)heads, a.queries = (uint16_t)queries;
  a.q_type = (uint8_t)q_type, a.out_type = (uint8_t)out_type;
  hipStream_t st = (hipStream_t)stream;
  return a.c.dim == 64    ? launch_groups<64>(a, rows, st)
         : a.c.dim == 128 ? launch_groups<128>(a, rows, st)
                          : launch_groups<256>(a, rows, st);
}
