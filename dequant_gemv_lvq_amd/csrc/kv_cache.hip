// The 4-bit key/value cache: storing tokens (lvq_kv_append, with the position
// rotation of q and k on the way) and reading them back (lvq_kv_read).
//
//   rotation   a' = a cos - b sin, b' = b cos + a sin over pairs of channels, every
//              product rounded to fp32 before the sum (no fused multiply-add), so that the
//              codes are those of the same formula in any fp32 program
//   4 bits     per token, head and group of channels: s = fp16((max - min) / 15),
//              l = fp16(min), code = clamp(rne((v - l) / s), 0, 15), value = s code + l
//
// Both are streams: a few operations per value, but two dependent reads (position, then
// page) before a store knows its place.  8192 tokens of 32 query and 8 key/value heads of 128
// channels: storing moves 181 MB in 45 us (4.0 TB/s, of a copy's 4.8), the waves waiting for
// memory for two thirds of it; reading back 42 MB in 15 us, of which 2 to 3 are a launch's.
// Tokens of one step are a launch each way, 3.7 and 4.2 us.

#include "kv_cache.h"

namespace lvq {

constexpr int kNoRotation = 0, kHalves = 1, kPairs = 2;

// ---------------------------------------------------------------- values

__device__ __forceinline__ float kv_bf16(uint32_t b) { return __builtin_bit_cast(float, b << 16); }

// Eight adjacent values as they lie in memory (any alignment of the type).
struct Raw8 {
  uint4 q[2];
};
__device__ __forceinline__ Raw8 raw8(const void* row, int type, int c) {
  Raw8 r;
  if (type == LVQ_F32) __builtin_memcpy(&r, (const uint8_t*)row + (size_t)c * 4, 32);
  else __builtin_memcpy(&r.q[0], (const uint8_t*)row + (size_t)c * 2, 16);
  return r;
}
__device__ __forceinline__ void widen(const Raw8& r, int type, float (&v)[8]) {
  const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w,
                         r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
  if (type == LVQ_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_bit_cast(float, w[i]);
  } else if (type == LVQ_F16) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i >> 1] >> (16 * (i & 1))));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = kv_bf16((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
  }
}

// Eight values to `type` (fp32, fp16 or bf16), rounded once to the nearest even.
__device__ __forceinline__ void store8(void* row, int type, int c, const float (&v)[8]) {
  if (type == LVQ_F32) {
    __builtin_memcpy((float*)row + c, v, 32);
    return;
  }
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (type == LVQ_F16)
      b[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i + 1]) << 16;
    else
      b[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i + 1]) << 16;
  }
  __builtin_memcpy((uint16_t*)row + c, b, 16);
}

// A result rounded to fp32 here: the instruction that multiplies or adds and rounds
// to fp16 at once would skip that rounding.
__device__ __forceinline__ float rounded(float v) {
  asm("" : "+v"(v));
  return v;
}

// x c - y s and x c + y s, the products rounded before the sum.
__device__ __forceinline__ float minus_products(float x, float c, float y, float s) {
#pragma clang fp contract(off)
  const float p = x * c, q = y * s;
  return rounded(p - q);
}
__device__ __forceinline__ float plus_products(float x, float c, float y, float s) {
#pragma clang fp contract(off)
  const float p = x * c, q = y * s;
  return rounded(p + q);
}

struct AppendArgs {
  KvPages c;
  uint16_t heads, rot;
  const void *q, *k, *v;
  const float *cos, *sin;
  const int32_t *seq, *pos;
  void* q_out;
  int q_stride, k_stride, v_stride;  // values
  int tokens, positions;
  uint8_t type, q_type, style;
};

// Threads of a workgroup: 16 tokens of dim / 8 lanes, four waves at least.
__host__ __device__ constexpr int append_threads(int dim) { return dim <= 128 ? 256 : 2 * dim; }
// Threads that rotate q, 16 channels each.
__host__ __device__ inline uint32_t q_threads(int tokens, int heads, int dim) {
  return (uint32_t)tokens * heads * (dim / 16);
}
__host__ __device__ inline uint32_t q_workgroups(int tokens, int heads, int dim) {
  const uint32_t n = append_threads(dim);
  return (q_threads(tokens, heads, dim) + n - 1) / n;
}

// Angles 8 u .. 8 u + 7 of a position (of a position past the table: of its last or none).
__device__ __forceinline__ size_t angle_row(const AppendArgs& a, int pos) {
  const int p = pos < 0 ? 0 : pos < a.positions ? pos : a.positions - 1;
  return (size_t)p * (a.rot / 2);
}
__device__ __forceinline__ void angles(const AppendArgs& a, int pos, int u, float (&c)[8],
                                       float (&s)[8]) {
  if (a.positions == 0) return;
  const size_t at = angle_row(a, pos) + 8 * u;
  __builtin_memcpy(c, a.cos + at, 32);
  __builtin_memcpy(s, a.sin + at, 32);
}

// Sequence and position of a token, and its page; -1 where it is to be left out.
struct Where {
  int seq, pos;
};
__device__ __forceinline__ Where ask(const AppendArgs& a, int token) {
  return {a.seq ? a.seq[token] : token, a.pos[token]};
}
__device__ __forceinline__ int find(const AppendArgs& a, Where w) {
  return a.rot && w.pos >= a.positions ? -1 : kv_page(a.c, w.seq, w.pos);
}

// q: a thread turns 16 channels of a head, two chunks of eight that belong together.
template <int DIM>
__device__ __forceinline__ void rotate_q(const AppendArgs& a) {
  constexpr uint32_t kPerHead = DIM / 16;
  const uint32_t per = a.heads * kPerHead;
  // the workgroup's first token by a division, the thread's from there: below 2^20 a float's
  // quotient of whole numbers, half a unit off the borders, is never off
  const uint32_t first = blockIdx.x * (uint32_t)append_threads(DIM), token0 = first / per;
  const uint32_t in = first - token0 * per + threadIdx.x;
  const uint32_t more = (uint32_t)(((float)in + 0.5f) * (1.f / (float)per));
  const int token = (int)(token0 + more);
  if (token >= a.tokens) return;
  // the place and the values are asked for together, then the angles and the page
  const Where at = ask(a, token);
  const uint32_t r = in - more * per;
  const int head = (int)(r / kPerHead), u = (int)(r % kPerHead);
  const bool turned = u * 16 < a.rot;
  const int base = head * DIM;
  const bool halves = turned && a.style == kHalves;
  const int c0 = base + (halves ? 8 * u : 16 * u);
  const int c1 = halves ? c0 + a.rot / 2 : c0 + 8;
  const uint8_t* row = (const uint8_t*)a.q + (int64_t)token * a.q_stride * (a.type == LVQ_F32 ? 4 : 2);
  const Raw8 r0 = raw8(row, a.type, c0), r1 = raw8(row, a.type, c1);
  float c[8], s[8];
  if (turned) angles(a, at.pos, u, c, s);
  if (find(a, at) < 0) return;
  float x[8], y[8];
  widen(r0, a.type, x);
  widen(r1, a.type, y);
  if (turned) {
    if (halves) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = x[j], q = y[j];
        x[j] = minus_products(p, c[j], q, s[j]);
        y[j] = plus_products(q, c[j], p, s[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p = x[2 * j], q = x[2 * j + 1];
        x[2 * j] = minus_products(p, c[j], q, s[j]);
        x[2 * j + 1] = plus_products(q, c[j], p, s[j]);
        p = y[2 * j], q = y[2 * j + 1];
        y[2 * j] = minus_products(p, c[4 + j], q, s[4 + j]);
        y[2 * j + 1] = plus_products(q, c[4 + j], p, s[4 + j]);
      }
    }
  }
  uint8_t* out = (uint8_t*)a.q_out +
                 (size_t)token * a.heads * DIM * (a.q_type == LVQ_F32 ? 4 : 2);
  store8(out, a.q_type, c0, x);
  store8(out, a.q_type, c1, y);
}

// Smallest (or, of the negated values, largest) over aligned groups of 4..32 lanes.
template <int CTRL>
__device__ __forceinline__ float dpp_min(float v) {
  const int i = __builtin_bit_cast(int, v);
  return fminf(v, __builtin_bit_cast(
                      float, __builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, false)));
}
__device__ __forceinline__ float lanes_min(float v, int lanes) {
  v = dpp_min<0xB1>(v);                    // quad_perm [1,0,3,2]
  v = dpp_min<0x4E>(v);                    // quad_perm [2,3,0,1]
  if (lanes >= 8) v = dpp_min<0x141>(v);   // row_half_mirror
  if (lanes >= 16) v = dpp_min<0x140>(v);  // row_mirror
  if (lanes >= 32) v = fminf(v, __shfl_xor(v, 16, kWave));
  return v;
}

// Eight values of a group spread over `lanes` lanes -> eight codes, each plus kCodeBias, and
// the group's scale and low end (fp16 bits, scale in the low half).  A NaN makes the
// smallest value minus infinity; with an infinity the scale is infinite, and reads as NaN.
constexpr uint32_t kCodeBias = 0x4B400000u;  // 1.5 * 2^23: a sum with it is rounded to a whole number
__device__ __forceinline__ uint32_t to_codes(const float (&v)[8], int lanes, uint32_t (&code)[8]) {
#pragma clang fp contract(off)
  float least = v[0], most = v[0], sum = v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    least = fminf(least, v[i]);
    most = fmaxf(most, v[i]);
    sum += v[i];
  }
  if (sum != sum) least = -__builtin_inff();
  least = lanes_min(least, lanes);
  most = -lanes_min(-most, lanes);
  const _Float16 s = (_Float16)rounded((most - least) * (1.f / 15.f));
  const _Float16 l = (_Float16)least;
  const float sf = (float)s, lf = (float)l;
  const float per = sf > 0.f ? 1.f / sf : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = rounded((v[i] - lf) * per);
    code[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(d, 0.f, 15.f) +
                                               __builtin_bit_cast(float, kCodeBias));
  }
  return (uint32_t)__builtin_bit_cast(uint16_t, s) |
         (uint32_t)__builtin_bit_cast(uint16_t, l) << 16;
}

// Keys or values of one head of 16 tokens: dim / 8 lanes per token, eight channels each.
template <int DIM>
__device__ __forceinline__ void store_kv(const AppendArgs& a, int block, uint8_t* tile) {
  constexpr int dim = DIM, lanes = dim / 8;
  const int per_tile = 2 * a.c.kv_heads;
  const int t = block / per_tile, which = block - t * per_tile;
  const bool values = which >= a.c.kv_heads;
  const int head = values ? which - a.c.kv_heads : which;
  const int i = threadIdx.x / lanes, lane = threadIdx.x - i * lanes;
  // tiles begin where the first token's block begins, so that those inside one
  // long run of positions are whole blocks
  const int shift = a.tokens > kBlockTokens ? a.pos[0] & (kBlockTokens - 1) : 0;
  const int token = t * kBlockTokens - shift + i;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  const int e = 8 * lane;
  int pos = 0, page = -1;
  // with 64 channels half of the threads have no token
  if (i < kBlockTokens && token >= 0 && token < a.tokens) {
    const Where where = ask(a, token);
    pos = where.pos;
    const int64_t step = (int64_t)token * (a.type == LVQ_F32 ? 4 : 2);
    const uint8_t* row = values ? (const uint8_t*)a.v + step * a.v_stride
                                : (const uint8_t*)a.k + step * a.k_stride;
    const bool turned = !values && e < a.rot, halves = a.style == kHalves;
    const bool first = e < a.rot / 2;  // of the two halves
    const int partner = turned && halves ? (first ? e + a.rot / 2 : e - a.rot / 2) : e;
    const Raw8 own = raw8(row, a.type, head * dim + e);
    const Raw8 other = raw8(row, a.type, head * dim + partner);
    float c[8], s[8], o[8];
    if (turned && halves) {
      angles(a, pos, (first ? e : partner) / 8, c, s);
    } else if (turned && a.positions) {
      const size_t at = angle_row(a, pos) + e / 2;
      __builtin_memcpy(c, a.cos + at, 16);
      __builtin_memcpy(s, a.sin + at, 16);
    }
    page = find(a, where);
    widen(own, a.type, v);
    if (turned && halves) {
      widen(other, a.type, o);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = first ? minus_products(v[j], c[j], o[j], s[j])
                     : plus_products(v[j], c[j], o[j], s[j]);
    } else if (turned) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = v[2 * j], q = v[2 * j + 1];
        v[2 * j] = minus_products(p, c[j], q, s[j]);
        v[2 * j + 1] = plus_products(q, c[j], p, s[j]);
      }
    }
  }
  const bool there = page >= 0;
  uint32_t code[8];
  const int group_shift = __builtin_ctz(lanes) - __builtin_ctz(a.c.groups);
  const uint32_t meta = to_codes(v, 1 << group_shift, code);
  const int in = pos & (kBlockTokens - 1);
  uint8_t* at = there ? kv_block(a.c, page, head, pos) : nullptr;
  if (there && (lane & ((1 << group_shift) - 1)) == 0)
    *(uint32_t*)(at + 16 * dim + (values ? 64 * a.c.groups : 0) + 64 * (lane >> group_shift) +
                 4 * in) = meta;
  if (!values) {
    // channel 8 lane + j is field j/2 + 4 (j%2) of word lane/4 of quarter lane%4
    uint32_t w = 0;  // modulo 2^32 the biases are one constant
#pragma unroll
    for (int j = 0; j < 8; ++j) w += (code[j] - kCodeBias) << (4 * (j / 2) + 16 * (j % 2));
    if (there) *(uint32_t*)(at + in * (dim / 2) + (lane & 3) * (dim / 8) + (lane >> 2) * 4) = w;
    return;
  }
  // channels 32 g + p (low half) and 32 g + 16 + p (high half) share a byte: lanes 0, 1 of a
  // quad hold low halves, 2 and 3 the high halves of the same pairs
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    lo += (code[j] - kCodeBias) << (8 * j);
    hi += (code[4 + j] - kCodeBias) << (8 * j);
  }
  const uint32_t other_lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)lo, 0x4E, 0xF, 0xF, false);
  const uint32_t other_hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)hi, 0x4E, 0xF, 0xF, false);
  // lanes 0, 1 take their first four pairs, lanes 2, 3 the last four of the same eight
  const bool upper = lane & 2;
  const uint32_t bytes = upper ? (other_hi | hi << 4) : (lo | other_lo << 4);
  const int pair = 16 * (lane >> 2) + 8 * (lane & 1) + (upper ? 4 : 0);
  // a whole block: its 16 tokens side by side
  __shared__ uint64_t first;
  if (threadIdx.x == 0) first = (uint64_t)at;
  __syncthreads();
  if (__syncthreads_and(i >= kBlockTokens || (there && in == i && (uint64_t)at == first))) {
    if (i < kBlockTokens)
#pragma unroll
      for (int j = 0; j < 4; ++j) tile[(pair + j) * kBlockTokens + i] = (uint8_t)(bytes >> (8 * j));
    __syncthreads();
    if ((int)threadIdx.x < dim / 2)
      *(uint4*)((uint8_t*)first + 8 * dim + threadIdx.x * 16) = ((const uint4*)tile)[threadIdx.x];
  } else if (there) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      at[8 * dim + (pair + j) * kBlockTokens + in] = (uint8_t)(bytes >> (8 * j));
  }
}

template <int DIM>
__global__ void __launch_bounds__(append_threads(DIM)) kv_append_kernel(AppendArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[DIM / 2 * kBlockTokens];
  const uint32_t rotating = q_workgroups(a.tokens, a.heads, DIM);
  if (blockIdx.x < rotating) rotate_q<DIM>(a);
  else store_kv<DIM>(a, (int)(blockIdx.x - rotating), tile);
}

// ---------------------------------------------------------------- reading back

struct ReadArgs {
  KvPages c;
  const int32_t *seq, *pos;
  void *k_out, *v_out;
  int tokens;
  uint8_t type;
};

// H: heads of a workgroup.  It waits for positions, then pages, then the cache: where tokens are
// many, four heads' loads are on their way at once; where few, one, so that more workgroups share
// the work.  us in a graph with one and with four, 8 heads of 128 channels: 1024 tokens 4.7, 7.0;
// 2048 6.3, 7.7; 4096, where the rule changes, 9.9, 9.5; 8192 17.3, 14.8; 16384 29.6, 23.9.  8 heads
// of 64: 4096 8.1, 8.0; 8192 13.0, 10.0.  2 heads of 256: 8192 12.2, 12.3; 16384, where it changes
// there, 22.4, 21.0.
constexpr int kReadHeads = 4;
inline int heads_at_once(const KvPages& c, long long tiles) {
  return tiles * c.kv_heads >= 8LL * device_cus() ? kReadHeads : 1;
}

// Keys or values of H heads of 16 tokens, eight channels per thread.  The values of a
// whole block come in as it lies and are turned in LDS; of others, byte by byte.
template <int DIM, int H>
__global__ void __launch_bounds__(append_threads(DIM)) kv_read_kernel(ReadArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[H][DIM / 2 * kBlockTokens];
  __shared__ uint64_t block0;
  constexpr int dim = DIM, lanes = dim / 8;
  const int per_kind = (a.c.kv_heads + H - 1) / H;
  const int per_tile = per_kind * (a.k_out && a.v_out ? 2 : 1);
  const int t = blockIdx.x / per_tile, which = blockIdx.x - t * per_tile;
  const bool values = !a.k_out || which >= per_kind;
  const int head0 = (a.k_out && values ? which - per_kind : which) * H;
  const int heads = a.c.kv_heads - head0 < H ? a.c.kv_heads - head0 : H;
  const int i = threadIdx.x / lanes, lane = threadIdx.x - i * lanes;
  // tiles begin where the first token's block begins, as where they are stored
  const int shift = a.tokens > kBlockTokens ? a.pos[0] & (kBlockTokens - 1) : 0;
  const int token = t * kBlockTokens - shift + i;
  const bool mine = i < kBlockTokens && token >= 0 && token < a.tokens;
  int pos = 0, page = -1;
  if (mine) {
    pos = a.pos[token];
    page = kv_page(a.c, a.seq ? a.seq[token] : token, pos);
  }
  const bool there = page >= 0;
  const int in = pos & (kBlockTokens - 1);
  const int group = lane >> (__builtin_ctz(lanes) - __builtin_ctz(a.c.groups));
  const uint8_t* const at0 = there ? kv_block(a.c, page, head0, pos) : nullptr;
  const int64_t next_head =
      (int64_t)(kv_block_bytes(dim, a.c.groups)) << (a.c.page_shift - 4);
  uint32_t m[H], w[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    m[h] = w[h] = 0;
    if (!there || h >= heads) continue;
    const uint8_t* at = at0 + h * next_head;
    m[h] = *(const uint32_t*)(at + 16 * dim + (values ? 64 * a.c.groups : 0) + 64 * group + 4 * in);
    if (!values)
      w[h] = *(const uint32_t*)(at + in * (dim / 2) + (lane & 3) * (dim / 8) + (lane >> 2) * 4);
  }
  bool whole = false;
  if (values) {
    if (threadIdx.x == 0) block0 = (uint64_t)at0;
    __syncthreads();
    whole = __syncthreads_and(i >= kBlockTokens || (there && in == i && (uint64_t)at0 == block0));
    if (whole) {
      for (int n = threadIdx.x; n < heads * (dim / 2); n += append_threads(dim)) {
        const int h = n / (dim / 2), pair = n - h * (dim / 2);
        ((uint4*)tile[h])[pair] =
            *(const uint4*)((const uint8_t*)block0 + h * next_head + 8 * dim + pair * 16);
      }
      __syncthreads();
    }
  }
  if (!mine) return;
  uint8_t* out = (uint8_t*)(values ? a.v_out : a.k_out) +
                 (size_t)token * a.c.kv_heads * dim * (a.type == LVQ_F32 ? 4 : 2);
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (h >= heads) break;
    const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)m[h]);
    const float l = (float)__builtin_bit_cast(_Float16, (uint16_t)(m[h] >> 16));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t code;
      if (!values) {
        code = w[h] >> (4 * (j / 2) + 16 * (j % 2));
      } else {
        const int byte = (16 * (lane >> 2) + 8 * (lane & 1) + j) * kBlockTokens + in;
        uint32_t b = 0;
        if (whole) b = tile[h][byte];
        else if (there) b = at0[h * next_head + 8 * dim + byte];
        code = b >> (lane & 2 ? 4 : 0);
      }
      v[j] = there ? rounded(__builtin_fmaf((float)(code & 15), s, l)) : 0.f;
    }
    store8(out, a.type, (head0 + h) * dim + 8 * lane, v);
  }
}

// ---------------------------------------------------------------- checks

int kv_pages(const lvq_kv_cache* c, KvPages* p) {
  if (!c) return LVQ_E_NULL;
  if (!kv_dim_ok(c->dim) || !kv_group_ok(c->dim, c->group) || !kv_page_ok(c->page) ||
      c->kv_heads < 1 || c->kv_heads > kKvMaxHeads || c->pages < 0 || c->seqs < 0 ||
      c->max_pages < 0)
    return LVQ_E_SHAPE;
  // positions, and sums of a few of them, are 32-bit
  if ((int64_t)c->max_pages * c->page > (1 << 30)) return LVQ_E_SHAPE;
  if ((c->pages && !c->pool) || (c->seqs && c->max_pages && !c->table)) return LVQ_E_NULL;
  if (!aligned16(c->pool) || !aligned16(c->table)) return LVQ_E_ALIGN;
  p->pool = (uint8_t*)c->pool, p->table = c->table, p->pages = c->pages;
  p->seqs = c->seqs, p->max_pages = c->max_pages;
  p->kv_heads = (uint16_t)c->kv_heads, p->dim = (uint16_t)c->dim;
  p->groups = (uint8_t)(c->group ? c->dim / c->group : 1);
  p->page_shift = (uint8_t)__builtin_ctz(c->page);
  return LVQ_OK;
}

inline size_t kv_type_bytes(int t) { return t == LVQ_F32 ? 4 : 2; }
inline bool kv_float(int t) { return t == LVQ_F32 || t == LVQ_F16 || t == LVQ_BF16; }

struct KvRange {
  const void* p;
  size_t n;
};

}  // namespace lvq

using namespace lvq;

extern "C" size_t lvq_kv_page_bytes(int kv_heads, int dim, int page, int group) {
  if (!kv_dim_ok(dim) || !kv_group_ok(dim, group) || !kv_page_ok(page) || kv_heads < 1 ||
      kv_heads > kKvMaxHeads)
    return 0;
  return (size_t)kv_heads * (page / kBlockTokens) * kv_block_bytes(dim, group ? dim / group : 1);
}

extern "C" int lvq_kv_append(const lvq_kv_cache* cache, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, int type, const int32_t* seq,
                             const int32_t* pos, int tokens, const float* cos, const float* sin,
                             int rot, int positions, int interleaved, const void* q,
                             int64_t q_stride, int heads, void* q_out, int q_out_type,
                             void* stream) {
  AppendArgs a;
  const int e = kv_pages(cache, &a.c);
  if (e) return e;
  const int dim = cache->dim;
  if (tokens < 0 || !kv_float(type) || heads < 0 || heads > kKvMaxHeads || rot < 0 || rot > dim ||
      rot % 16 || positions < 0 || interleaved < 0 || interleaved > 1)
    return LVQ_E_SHAPE;
  if (heads && q_out_type != LVQ_F16 && q_out_type != LVQ_BF16 && q_out_type != LVQ_F32)
    return LVQ_E_SHAPE;
  const int64_t kv_cols = (int64_t)cache->kv_heads * dim, q_cols = (int64_t)heads * dim;
  if (k_stride < kv_cols || v_stride < kv_cols || (heads && q_stride < q_cols) ||
      k_stride > INT32_MAX || v_stride > INT32_MAX || (heads && q_stride > INT32_MAX))
    return LVQ_E_SHAPE;
  if (!seq && tokens > cache->seqs) return LVQ_E_SHAPE;
  if (tokens == 0) return LVQ_OK;
  // an empty table of angles may have no address: every position is past it
  if (!k || !v || !pos || (rot && positions && (!cos || !sin)) || (heads && (!q || !q_out)))
    return LVQ_E_NULL;
  const size_t tb = kv_type_bytes(type);
  if ((uintptr_t)k % tb || (uintptr_t)v % tb || (heads && (uintptr_t)q % tb) ||
      (uintptr_t)seq % 4 || (uintptr_t)pos % 4 || !aligned16(cos) || !aligned16(sin) ||
      !aligned16(q_out))
    return LVQ_E_ALIGN;
  auto span = [&](int64_t stride, int64_t cols) {
    return ((size_t)(tokens - 1) * stride + cols) * tb;
  };
  const size_t turn = (size_t)positions * (rot / 2) * 4;
  const KvRange in[8] = {{k, span(k_stride, kv_cols)},
                         {v, span(v_stride, kv_cols)},
                         {heads ? q : nullptr, heads ? span(q_stride, q_cols) : 0},
                         {cos, turn},
                         {sin, turn},
                         {seq, (size_t)tokens * 4},
                         {pos, (size_t)tokens * 4},
                         {a.c.table, kv_table_bytes(a.c)}};
  const KvRange made[2] = {{a.c.pool, kv_pool_bytes(a.c)},
                           {heads ? q_out : nullptr,
                            (size_t)tokens * q_cols * (heads ? kv_type_bytes(q_out_type) : 0)}};
  for (const KvRange& m : made)
    for (const KvRange& r : in)
      if (ranges_overlap(m.p, m.n, r.p, r.n)) return LVQ_E_SHAPE;
  if (ranges_overlap(made[0].p, made[0].n, made[1].p, made[1].n)) return LVQ_E_SHAPE;
  a.q = q, a.k = k, a.v = v;
  a.q_stride = heads ? (int)q_stride : 0, a.k_stride = (int)k_stride, a.v_stride = (int)v_stride;
  a.cos = cos, a.sin = sin, a.seq = seq, a.pos = pos, a.q_out = q_out;
  a.tokens = tokens, a.positions = positions, a.heads = (uint16_t)heads;
  a.rot = (uint16_t)rot, a.type = (uint8_t)type, a.q_type = (uint8_t)q_out_type;
  a.style = rot == 0 ? kNoRotation : interleaved ? kPairs : kHalves;
  // the kernel counts threads and workgroups in 32 bits
  const long long tiles = (tokens + kBlockTokens - 1LL) / kBlockTokens + (tokens > kBlockTokens);
  if ((long long)tokens * heads * (dim / 16) >= INT32_MAX - 512 ||
      tiles * 2 * cache->kv_heads >= INT32_MAX / 4)
    return LVQ_E_SHAPE;
  const unsigned all = q_workgroups(tokens, heads, dim) + (unsigned)(tiles * 2 * cache->kv_heads);
  clear_hip_error();
  const dim3 grid(all), threads(append_threads(dim));
  hipStream_t st = (hipStream_t)stream;
  if (dim == 64) hipLaunchKernelGGL(kv_append_kernel<64>, grid, threads, 0, st, a);
  else if (dim == 128) hipLaunchKernelGGL(kv_append_kernel<128>, grid, threads, 0, st, a);
  else hipLaunchKernelGGL(kv_append_kernel<256>, grid, threads, 0, st, a);
  return launch_status();
}

extern "C" int lvq_kv_read(const lvq_kv_cache* cache, const int32_t* seq, const int32_t* pos,
                           int tokens, void* k_out, void* v_out, int out_type, void* stream) {
  ReadArgs a;
  const int e = kv_pages(cache, &a.c);
  if (e) return e;
  if (tokens < 0 || !kv_float(out_type) || (!seq && tokens > cache->seqs)) return LVQ_E_SHAPE;
  if (tokens == 0 || (!k_out && !v_out)) return LVQ_OK;
  if (!pos) return LVQ_E_NULL;
  if ((uintptr_t)seq % 4 || (uintptr_t)pos % 4 || !aligned16(k_out) || !aligned16(v_out))
    return LVQ_E_ALIGN;
  const size_t n = (size_t)tokens * cache->kv_heads * cache->dim * kv_type_bytes(out_type);
  const KvRange in[4] = {{a.c.pool, kv_pool_bytes(a.c)},
                         {a.c.table, kv_table_bytes(a.c)},
                         {seq, (size_t)tokens * 4},
                         {pos, (size_t)tokens * 4}};
  for (const void* o : {(const void*)k_out, (const void*)v_out})
    for (const KvRange& r : in)
      if (ranges_overlap(o, n, r.p, r.n)) return LVQ_E_SHAPE;
  if (ranges_overlap(k_out, n, v_out, n)) return LVQ_E_SHAPE;
  a.seq = seq, a.pos = pos, a.k_out = k_out, a.v_out = v_out;
  a.tokens = tokens, a.type = (uint8_t)out_type;
  const long long tiles = (tokens + kBlockTokens - 1LL) / kBlockTokens + (tokens > kBlockTokens);
  const int kinds = k_out && v_out ? 2 : 1, at_once = heads_at_once(a.c, tiles);
  if (tiles * cache->kv_heads * kinds >= INT32_MAX / 4) return LVQ_E_SHAPE;
  const dim3 grid((unsigned)(tiles * kinds * ((cache->kv_heads + at_once - 1) / at_once)));
  const dim3 threads(append_threads(cache->dim));
  hipStream_t st = (hipStream_t)stream;
  clear_hip_error();
  auto launch = [&](auto one, auto many) {
    if (at_once == 1) hipLaunchKernelGGL(one, grid, threads, 0, st, a);
    else hipLaunchKernelGGL(many, grid, threads, 0, st, a);
  };
  if (cache->dim == 64) launch(kv_read_kernel<64, 1>, kv_read_kernel<64, kReadHeads>);
  else if (cache->dim == 128) launch(kv_read_kernel<128, 1>, kv_read_kernel<128, kReadHeads>);
  else launch(kv_read_kernel<256, 1>, kv_read_kernel<256, kReadHeads>);
  return launch_status();
}
