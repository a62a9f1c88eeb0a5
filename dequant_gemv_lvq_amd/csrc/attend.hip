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
// A wave takes 64 tokens at a time, four blocks of 16.  Keys: four 16x16 products (rows
// by tokens) of dim / 32 steps; lane 16 b + t then holds token t of block b and four
// rows (with 4 or 8 rows the 16 of the product repeat them, and every lane keeps what is
// its own).  The weights p pass through LDS to become operands again: product of the
// values' channels by rows.  Workgroups of four waves split a sequence further, and a
// second launch joins their parts (flash decoding).

#include "kv_cache.h"

namespace lvq {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttWaves = 4;
constexpr int kAttTokens = 64;  // of a wave at a time
constexpr uint32_t kCodeMask = 0x03C003C0u;
constexpr float kCodeUnit = 0x1p18f;
constexpr int kPStride = 144;   // bytes of a row of weights in LDS: 64 fp16 and 16 to spread banks

struct AttArgs {
  KvPages c;
  uint16_t heads, queries;
  const int32_t* lens;
  const void* q;
  void* out;
  float* parts;   // [seqs][kv_heads][splits][rows][dim], then {maximum, sum} of each
  int64_t q_stride;  // values
  float scale;    // of the logits, in powers of two
  int window, splits;
  uint16_t tiles;  // of rows
  uint8_t q_type, out_type;
};
static_assert(sizeof(AttArgs) < 128, "launches of 128 bytes and more are slower");

// What a sequence's workgroups share: the tokens any of its queries sees, in units of 64.
struct Span {
  int first, last;   // blocks of 64 tokens [first, last)
  int parts, each;   // workgroups, and blocks of each
  int len;
};
__device__ __forceinline__ Span att_span(const KvPages& c, int len, int queries, int window,
                                         int splits) {
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
  const int n = s.last - s.first;
  int parts = (n + kAttWaves - 1) / kAttWaves;
  parts = parts < splits ? parts : splits;
  parts = parts < 1 ? 1 : parts;
  s.each = (n + parts - 1) / parts;
  s.parts = s.each ? (n + s.each - 1) / s.each : 1;
  return s;
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

// Over the lanes that hold the same rows: the 16 of a quarter, and the quarters
// RT / 4 apart.
template <int RT>
__device__ __forceinline__ float rows_max(float v) {
  v = dpp_max_f<0xB1>(v);
  v = dpp_max_f<0x4E>(v);
  v = dpp_max_f<0x141>(v);
  v = dpp_max_f<0x140>(v);
  if constexpr (RT <= 4) v = fmaxf(v, __shfl_xor(v, 16, kWave));
  if constexpr (RT <= 8) v = fmaxf(v, __shfl_xor(v, 32, kWave));
  return v;
}
template <int RT>
__device__ __forceinline__ float rows_sum(float v) {
  v = dpp_add<0xB1, 0xF>(v);
  v = dpp_add<0x4E, 0xF>(v);
  v = dpp_add<0x141, 0xF>(v);
  v = dpp_add<0x140, 0xF>(v);
  if constexpr (RT <= 4) v += __shfl_xor(v, 16, kWave);
  if constexpr (RT <= 8) v += __shfl_xor(v, 32, kWave);
  return v;
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

// LDS: while the tokens are read, each wave's weights (2 RT rows); then, in the same
// place, each wave's part of the result [RT][DIM], maxima, sums and low ends.
constexpr int att_p_bytes(int RT) { return 2 * RT * kPStride; }
constexpr int att_part_bytes(int RT, int dim) { return RT * dim * 4; }
constexpr int att_wave_bytes(int RT, int dim, int groups) {
  const int small = (2 + groups) * RT * 4;
  const int a = att_p_bytes(RT), b = att_part_bytes(RT, dim) + small;
  return (a > b ? a : b);
}

template <int DIM, int RT, int NG>
__global__ void __launch_bounds__(kAttWaves* kWave) attend_kernel(AttArgs a) {
  constexpr int KS = DIM / 32;       // steps of 32 channels
  constexpr int GS = KS / NG;        // of a group
  constexpr int NT = RT / 4;         // tokens of a lane
  __shared__ __attribute__((aligned(16))) uint8_t smem[kAttWaves][att_wave_bytes(RT, DIM, NG)];
  const int lane = threadIdx.x & (kWave - 1), t16 = lane & 15, quarter = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int seq = blockIdx.z, part = blockIdx.y;
  const int head = blockIdx.x / a.tiles, tile = blockIdx.x - head * a.tiles;
  const Span sp = att_span(a.c, a.lens[seq], a.queries, a.window, a.splits);
  if (part >= sp.parts) return;
  const int per = a.heads / a.c.kv_heads, rows = per * a.queries;
  const int row0 = tile * 16;
  const int b0 = sp.first + part * sp.each;
  const int b1 = b0 + sp.each < sp.last ? b0 + sp.each : sp.last;

  // q: operand row t16 (repeated every RT rows), channels 32 s + 8 quarter .. + 7 of step s
  half8_t qa[KS];
  float qs[NG][4], unit[4];  // of this lane's four rows: sums of q over a group, logit's unit
  int see_first[4], see_last[4];
  {
    const int r = row0 + (t16 & (RT - 1));
    const bool real = r < rows;
    const int query = real ? r / per : 0, h = head * per + (real ? r - query * per : 0);
    const uint16_t* row = (const uint16_t*)a.q +
                          ((int64_t)seq * a.queries + query) * a.q_stride + (int64_t)h * DIM;
    uint4 raw[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s)
      __builtin_memcpy(&raw[s], row + 32 * s + 8 * quarter, 16);
    float sum[NG], mine = a.scale * kCodeUnit;
#pragma unroll
    for (int g = 0; g < NG; ++g) sum[g] = 0.f;
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
          const uint32_t b = (i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
          v[s][i] = __builtin_bit_cast(float, b);
          const uint32_t m = b & 0x7F800000u;
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
      mine *= __builtin_bit_cast(float, top);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) qa[s][i] = (_Float16)(v[s][i] * down);
    }
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[s / GS] += (float)qa[s][i];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      sum[g] += __shfl_xor(sum[g], 16, kWave);
      sum[g] += __shfl_xor(sum[g], 32, kWave);
    }
    // from lanes by operand row to lanes by result row
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int from = 4 * (quarter & (NT - 1)) + i;
#pragma unroll
      for (int g = 0; g < NG; ++g) qs[g][i] = __shfl(sum[g], from, kWave) * (1.f / kCodeUnit);
      unit[i] = __shfl(mine, from, kWave);
      const int rr = row0 + from, qq = rr / per;
      see_last[i] = sp.len - a.queries + qq;
      see_first[i] = a.window > 0 ? see_last[i] - a.window + 1 : 0;
      if (rr >= rows) see_last[i] = sp.len - 1, see_first[i] = 0;  // not stored
    }
  }
  // tokens that every row sees
  int all_first, all_last;
  // and the first that any row sees
  const int any_first = a.window > 0 ? sp.len - a.queries - a.window + 1 : 0;
  {
    const int q0 = row0 / per, q1 = (row0 + RT < rows ? row0 + RT - 1 : rows - 1) / per;
    all_last = sp.len - a.queries + q0;
    all_first = a.window > 0 ? sp.len - a.queries + q1 - a.window + 1 : 0;
  }

  uint8_t* const lds = smem[wv];
  const int64_t page_size = kv_page_size(a.c);
  constexpr int kBlock = kv_block_bytes(DIM, NG);
  const int blocks_mask = (1 << (a.c.page_shift - 4)) - 1;
  const int32_t* table = a.c.table + (int64_t)seq * a.c.max_pages;
  const uint8_t* pool = a.c.pool + (int64_t)head * (blocks_mask + 1) * kBlock;

  // the page of this lane's block (quarter) of 64 tokens
  auto page_of = [&](int b) {
    const int at = (b * kAttTokens + 16 * quarter) >> a.c.page_shift;
    return at < a.c.max_pages ? table[at] : -1;
  };
  struct Tokens {
    uint32_t k[4][KS];
    u32x4 v[KS];
    uint32_t ks[NG], vs[NG];
  };
  Tokens x;
  auto block_at = [&](int b, int page) {
    const bool bad = page < 0 || page >= a.c.pages;
    return pool + (bad ? 0 : page) * page_size +
           ((4 * b + quarter) & blocks_mask) * (int64_t)kBlock;
  };
  auto load_k = [&](const uint8_t* at) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)(uintptr_t)at, 16 * j);
      const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)((uintptr_t)at >> 32), 16 * j);
      const uint8_t* p = (const uint8_t*)((uint64_t)hi << 32 | lo) + (t16 * 4 + quarter) * KS * 4;
      __builtin_memcpy(x.k[j], p, KS * 4);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) x.ks[g] = *(const uint32_t*)(at + 16 * DIM + 64 * g + 4 * t16);
  };
  auto load_v = [&](const uint8_t* at) {
#pragma unroll
    for (int g = 0; g < NG; ++g)
      x.vs[g] = *(const uint32_t*)(at + 16 * DIM + 64 * (NG + g) + 4 * t16);
#pragma unroll
    for (int s = 0; s < KS; ++s) __builtin_memcpy(&x.v[s], at + 8 * DIM + (16 * s + t16) * 16, 16);
  };

  float m[4], l[4], low[NG][4];
  f32x4_t acc[KS][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -__builtin_inff(), l[i] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) low[g][i] = 0.f;
  }
#pragma unroll
  for (int s = 0; s < KS; ++s) acc[s][0] = acc[s][1] = f32x4_t{0, 0, 0, 0};
  // the weights' unit: 2^6 over a power of two at or above the largest scale so far
  float smax = 0.f, pu = 1.f;

  int b = b0 + wv;
  int page = b < b1 ? page_of(b) : -1;
  int page_next = b + kAttWaves < b1 ? page_of(b + kAttWaves) : -1;
  const uint8_t* at = block_at(b, page);
  if (b < b1) {
    load_k(at);
    load_v(at);
  }
  for (; b < b1; b += kAttWaves) {
    // ---- logits
    float x0[NT][4];
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
          d[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
              qa[s], codes8(w << 6, w << 2, w >> 2, w >> 6), d[j], 0, 0, 0);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4_t e;
        uint32_t sl;
        if constexpr (RT == 4) {
          e = quarter & 2 ? (quarter & 1 ? d[3] : d[2]) : (quarter & 1 ? d[1] : d[0]);
          sl = x.ks[g];
        } else if constexpr (RT == 8) {
          e = quarter & 2 ? d[2 * n + 1] : d[2 * n];
          sl = __shfl(x.ks[g], 16 * (2 * n + (quarter >> 1)) + t16, kWave);
        } else {
          e = d[n];
          sl = __shfl(x.ks[g], 16 * n + t16, kWave);
        }
        const float s = att_f16(sl), lo = att_f16(sl >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float r = __builtin_fmaf(s, e[i], lo * qs[g][i]);
          x0[n][i] = g ? x0[n][i] + r : r;
        }
      }
    }
    uint32_t vs[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) vs[g] = x.vs[g];
    // ---- what a row does not see
    const int t0 = b * kAttTokens;
    const bool bad = page < 0 || page >= a.c.pages;
    if (t0 < all_first || t0 + kAttTokens - 1 > all_last || __any(bad)) {
      // a value that is not finite: NaN in the rows that see it, and nothing in the others
      bool wild = false;
#pragma unroll
      for (int g = 0; g < NG; ++g)
        wild |= (vs[g] & 0x7C00u) == 0x7C00u || (vs[g] & 0x7C000000u) == 0x7C000000u;
      const int mine = t0 + 16 * quarter + t16;
      const bool none = bad || mine >= sp.len || mine < any_first;
      const int flags = (none ? 1 : 0) | (wild ? 2 : 0);
      if (none || wild)
#pragma unroll
        for (int g = 0; g < NG; ++g) vs[g] = 0;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int blk = RT == 4 ? quarter : RT == 8 ? 2 * n + (quarter >> 1) : n;
        const int tok = t0 + 16 * blk + t16;
        const int f = RT == 4 ? flags : __shfl(flags, 16 * blk + t16, kWave);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (f & 2) x0[n][i] = __builtin_nanf("");
          if ((f & 1) || tok < see_first[i] || tok > see_last[i]) x0[n][i] = -__builtin_inff();
        }
      }
    }
    // ---- the next tokens' keys
    const int bn = b + kAttWaves;
    const int page_n = page_next;
    const uint8_t* at_n = block_at(bn, page_n);
    if (bn < b1) {
      page_next = bn + kAttWaves < b1 ? page_of(bn + kAttWaves) : -1;
      load_k(at_n);
    }
    // ---- maxima: left behind by up to 2^8, so that they seldom change
    float top = 0.f;
    bool grown = false;
#pragma unroll
    for (int g = 0; g < NG; ++g) top = fmaxf(top, fabsf(att_f16(vs[g])));
    grown = top > smax;
    float xm[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xm[i] = x0[0][i];
#pragma unroll
      for (int n = 1; n < NT; ++n) xm[i] = fmaxf(xm[i], x0[n][i]);
      grown |= xm[i] * unit[i] > m[i] + 8.f;
    }
    if (__any(grown)) {
      float old_pu = pu;
      top = fmaxf(top, smax);
      top = rows_max<4>(top);
      smax = top;
      if (top > 0.f && top < __builtin_inff()) {
        // 2^6 over the power of two above it
        const uint32_t e = __builtin_bit_cast(uint32_t, top) & 0x7F800000u;
        pu = __builtin_bit_cast(float, 0x7F800000u + 0x02000000u - e);
      }
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float nm = fmaxf(m[i], rows_max<RT>(xm[i]) * unit[i]);
        f[i] = m[i] == nm ? 1.f : __builtin_amdgcn_exp2f(m[i] - nm);  // 0 from minus infinity
        m[i] = nm;
        l[i] *= f[i];
#pragma unroll
        for (int g = 0; g < NG; ++g) low[g][i] *= f[i];
        f[i] *= pu / old_pu;
      }
      // from lanes by four rows to lanes by one: row t16 is f[t16 % 4] of quarter t16 / 4
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float o = __shfl(f[i], 16 * ((t16 & (RT - 1)) >> 2), kWave);
        mine = (t16 & 3) == i ? o : mine;
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[s][h] *= mine;
    }
    // ---- weights
    float p[NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float mi = m[i] == -__builtin_inff() ? 0.f : m[i];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        p[n][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x0[n][i], unit[i], -mi));
        l[i] += p[n][i];
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      lds_order();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int blk = RT == 4 ? quarter : RT == 8 ? 2 * n + (quarter >> 1) : n;
        const uint32_t sl = RT == 4 ? vs[g] : __shfl(vs[g], 16 * blk + t16, kWave);
        const float s = att_f16(sl) * pu, lo = att_f16(sl >> 16);
        // the values' pairs hold tokens 0 and 2, 1 and 3 of four
        const int tok = 16 * blk + ((t16 & 12) | (t16 & 1) << 1 | (t16 & 2) >> 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          low[g][i] = __builtin_fmaf(p[n][i], lo, low[g][i]);
          const float w = p[n][i] * s;
          const _Float16 hi = (_Float16)w, rest = (_Float16)(w - (float)hi);
          const int row = 4 * (quarter & (NT - 1)) + i;
          *(_Float16*)(lds + row * kPStride + 2 * tok) = hi;
          *(_Float16*)(lds + (RT + row) * kPStride + 2 * tok) = rest;
        }
      }
      lds_order();
      // operand column t16: row t16 of the rounded weights, then of the rests
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = RT == 4 ? t16 & 7 : t16;
        const half8_t w0 = *(const half8_t*)(lds + col * kPStride + 32 * quarter + 16 * k);
        half8_t w1;
        if constexpr (RT == 16)
          w1 = *(const half8_t*)(lds + (RT + col) * kPStride + 32 * quarter + 16 * k);
#pragma unroll
        for (int s = g * GS; s < (g + 1) * GS; ++s) {
          const uint32_t c0 = x.v[s][2 * k], c1 = x.v[s][2 * k + 1];
          const half8_t lo = codes8(c0 << 6, c0 >> 2, c1 << 6, c1 >> 2);
          const half8_t hi = codes8(c0 << 2, c0 >> 6, c1 << 2, c1 >> 6);
          acc[s][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, w0, acc[s][0], 0, 0, 0);
          acc[s][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, w0, acc[s][1], 0, 0, 0);
          if constexpr (RT == 16) {
            acc[s][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, w1, acc[s][0], 0, 0, 0);
            acc[s][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, w1, acc[s][1], 0, 0, 0);
          }
        }
      }
    }
    if (bn < b1) load_v(at_n);
    page = page_n;
  }

  // ---- this wave's part: maxima, sums and low ends by row, then the result
  lds_order();
  float* const part_o = (float*)lds;
  float* const part_m = (float*)(lds + att_part_bytes(RT, DIM));
  float* const part_l = part_m + RT;
  float* const part_low = part_l + RT;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * (quarter & (NT - 1)) + i;
    const float sum = rows_sum<RT>(l[i]);
    if (t16 == 0 && quarter < NT) part_m[row] = m[i], part_l[row] = sum;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float v = rows_sum<RT>(low[g][i]);
      if (t16 == 0 && quarter < NT) part_low[g * RT + row] = v;
    }
  }
  lds_order();
  const float back = kCodeUnit / pu;
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4_t v = acc[s][h];
      if constexpr (RT < 16) {  // the rests' columns are RT further
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += __shfl(v[i], (lane + RT) & 63, kWave);
      }
      if (t16 < RT) {
        const float lo = part_low[(s / GS) * RT + t16];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(v[i], back, lo);
        *(f32x4_t*)(part_o + t16 * DIM + 32 * s + 16 * h + 4 * quarter) = v;
      }
    }
  __syncthreads();

  // ---- the workgroup's: four channels of a row per thread
  for (int at4 = threadIdx.x; at4 < RT * (DIM / 4); at4 += kAttWaves * kWave) {
    const int r = at4 / (DIM / 4), c = (at4 - r * (DIM / 4)) * 4;
    if (row0 + r >= rows) break;
    float big = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kAttWaves; ++w)
      big = fmaxf(big, ((float*)(smem[w] + att_part_bytes(RT, DIM)))[r]);
    float sum = 0.f;
    f32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kAttWaves; ++w) {
      const float* ml = (float*)(smem[w] + att_part_bytes(RT, DIM));
      const float f = ml[r] == big ? 1.f : __builtin_amdgcn_exp2f(ml[r] - big);
      sum = __builtin_fmaf(ml[RT + r], f, sum);
      v += *(const f32x4_t*)((float*)smem[w] + r * DIM + c) * f;
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
        ml[0] = big, ml[1] = sum;
      }
    }
  }
}

// Joins the parts of a row: a workgroup per row, its parts dealt to groups of DIM / 4
// threads, four channels per thread.
template <int DIM>
__global__ void __launch_bounds__(256) attend_join_kernel(AttArgs a) {
  constexpr int T = DIM / 4, N = 256 / T;
  __shared__ f32x4_t part[N][T];
  __shared__ float sums[N];
  const int per = a.heads / a.c.kv_heads, rows = per * a.queries;
  const int seq = blockIdx.y, head = blockIdx.x / rows, r = blockIdx.x - head * rows;
  const Span sp = att_span(a.c, a.lens[seq], a.queries, a.window, a.splits);
  if (sp.parts == 1) return;  // written by its only workgroup
  const size_t n = (size_t)rows * a.splits;
  const size_t at = ((size_t)seq * a.c.kv_heads + head) * n + r;
  const float* ml = a.parts + (size_t)a.c.seqs * a.c.kv_heads * n * DIM + 2 * at;
  const float* o = a.parts + at * DIM;
  float big = -__builtin_inff();
  for (int p = threadIdx.x & (kWave - 1); p < sp.parts; p += kWave)
    big = fmaxf(big, ml[(size_t)2 * p * rows]);
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) big = fmaxf(big, __shfl_xor(big, d, kWave));
  const int g = threadIdx.x / T, c = threadIdx.x - g * T;
  float sum = 0.f;
  f32x4_t v = {0, 0, 0, 0};
#pragma unroll 4
  for (int p = g; p < sp.parts; p += N) {
    const float mp = ml[(size_t)2 * p * rows];
    const float f = mp == big ? 1.f : __builtin_amdgcn_exp2f(mp - big);
    sum = __builtin_fmaf(ml[(size_t)2 * p * rows + 1], f, sum);
    f32x4_t w;
    __builtin_memcpy(&w, o + (size_t)p * rows * DIM + 4 * c, 16);
    v += w * f;
  }
  part[g][c] = v;
  if (c == 0) sums[g] = sum;
  __syncthreads();
  if (g == 0) {
    for (int k = 1; k < N; ++k) v += part[k][c], sum += sums[k];
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int query = r / per, h = head * per + r - query * per;
    att_store4(a.out, a.out_type,
               (((size_t)seq * a.queries + query) * a.heads + h) * DIM + 4 * c, v * inv);
  }
}

// ---------------------------------------------------------------- launch

// Workgroups that a sequence's tokens are split over, at most: enough to fill the chip
// about twice, and no more than there are tokens for.
inline int att_splits(const KvPages& c, int queries, int window, int tiles) {
  long long tokens = (long long)c.max_pages << c.page_shift;
  if (window > 0 && window + queries + kAttTokens < tokens)
    tokens = window + queries + kAttTokens;
  const long long most =
      (tokens + kAttTokens * kAttWaves - 1) / (kAttTokens * kAttWaves);
  const long long wgs = (long long)c.seqs * c.kv_heads * tiles;
  long long want = (6LL * device_cus() + wgs - 1) / (wgs > 0 ? wgs : 1);
  want = want < most ? want : most;
  return want < 1 ? 1 : (int)want;
}

inline size_t att_space(const KvPages& c, int heads, int queries, int splits) {
  return splits == 1 ? 0 : (size_t)c.seqs * heads * queries * splits * (c.dim + 2) * 4;
}

template <int DIM, int RT, int NG>
int launch_attend(const AttArgs& a, hipStream_t st) {
  const dim3 grid(a.c.kv_heads * a.tiles, a.splits, a.c.seqs), block(kAttWaves * kWave);
  clear_hip_error();
  hipLaunchKernelGGL((attend_kernel<DIM, RT, NG>), grid, block, 0, st, a);
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
                   att_splits(c, queries, 0, att_tiles(c, heads, queries)));
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
  a.splits = att_splits(a.c, queries, window, a.tiles);
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
  a.scale = scale * 1.44269504f, a.window = window;
  a.heads = (uint16_t)heads, a.queries = (uint16_t)queries;
  a.q_type = (uint8_t)q_type, a.out_type = (uint8_t)out_type;
  hipStream_t st = (hipStream_t)stream;
  return a.c.dim == 64    ? launch_groups<64>(a, rows, st)
         : a.c.dim == 128 ? launch_groups<128>(a, rows, st)
                          : launch_groups<256>(a, rows, st);
}
