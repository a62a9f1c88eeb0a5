// A mixture-of-experts layer in 4-bit weights for a few tokens (q4_moe).
//
//   l = R x, the `top` largest l are chosen, w = softmax(l) of the chosen
//   y = sum_e w_e D_e (silu(G_e x) * (U_e x))
//
// Three launches, each needing all of the one before: the router's logits (a workgroup per
// expert and four tokens), the choice and the chosen experts' gate and up products with the activation,
// the down products with the weighted sum.  The choice is a few hundred operations, so
// every workgroup of the second launch makes it for itself.
//
// The products are those of the 4-bit matvec: 4x4x4 matrix products in 16 blocks, lane l
// holding row l % 4 of a quad of rows and unit l / 4 of a step of 16 units of 32 columns; the
// codes are fp16 subnormals (bits 6..9 of the mantissa), scale and zero are applied in the
// lane in fp32.  Up to four tokens of an expert share a pass over its weights (a job).  x
// sits in LDS.  The activations between the products are kept as two fp16, the rounded
// value and the rest times 2^11 (22 bits), which the down product multiplies side by side.
//
// What bounds it, and what it measured (GPU, one call; 128 experts of 2048 x 768, 8 chosen):
// one token, the three launches and in each a few trips to memory (in a trace, router 2.9 us, gate
// and up 8.4 for 13 MB, of which about 2 for the choice, down 4.5 for 7 MB); sixteen tokens, the
// read of the weights and, in the down product, the instructions around it (4.7 us; 33 for
// 128 MB, 3.9 TB/s; 27 for 78 MB with the activations, 2.9 TB/s); four tokens through 8
// experts of 4096 x 12288 with zeros, 2 chosen, the read (4.7; 57 for 284 MB, 5.0 TB/s; 44
// for 145 MB, 3.3).

#include "q4_dev.h"

namespace lvq {

constexpr float kMoeUnit = 0x1p-18f;   // of a code inside an fp16
// Of an activation's rest: as large as the value was, so that it is a normal number where that is.
constexpr float kRestUnit = 0x1p11f;
constexpr int kGateWaves = 16;
constexpr int kMaxPairs = LVQ_MAX_MOE_TOKENS * LVQ_MAX_MOE_TOP;
constexpr int kMaxExperts = 512;

// ---------------------------------------------------------------- router

struct RouterArgs {
  const uint16_t* x;
  const void* router;
  float* logits;  // [tokens][experts], then as many rests
  int tokens, hidden, experts;
  int type;
};

// Sum over the 64 lanes of a wave, valid in lane 63, as wave_sum_lane63 adds them.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_add64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, CTRL, ROW_MASK, 0xF, false);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROW_MASK, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum64_lane63(double v) {
  v = dpp_add64<0xB1, 0xF>(v);
  v = dpp_add64<0x4E, 0xF>(v);
  v = dpp_add64<0x141, 0xF>(v);
  v = dpp_add64<0x140, 0xF>(v);
  v = dpp_add64<0x142, 0xA>(v);
  return dpp_add64<0x143, 0xC>(v);
}

// A workgroup: one expert, N tokens, a thread for eight columns (up to kRouterWaves of them, then
// in rounds), so that one trip to memory serves all.  The choice is between logits as close as they
// come, so they are summed in 64 bits (every product is exact there) and left as two floats, the
// rounded value and the rest.  In fp32, experts nearer than 2^-20 or so were chosen by the roundings;
// the sums cost 0.1 us of one token's layer of 15.
constexpr int kRouterWaves = 16;

template <int N>
__global__ void __launch_bounds__(kRouterWaves* kWave) moe_router_kernel(RouterArgs a) {
  __shared__ double red[kRouterWaves][N];
  const int e = blockIdx.x, t0 = blockIdx.y * N;
  const int n = a.tokens - t0 < N ? a.tokens - t0 : N;
  const size_t row = (size_t)e * a.hidden;
  double acc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) acc[k] = 0;
  for (int c = threadIdx.x * 8; c < a.hidden; c += blockDim.x * 8) {
    uint32_t r[8], x[N][4];
    // tokens past the last: the last again, not stored
    auto x_row = [&](int k) { return a.x + (size_t)(t0 + (k < n ? k : n - 1)) * a.hidden + c; };
    if (c + 8 <= a.hidden) {
      if (a.type == LVQ_F32) __builtin_memcpy(r, (const float*)a.router + row + c, 32);
      else __builtin_memcpy(r, (const uint16_t*)a.router + row + c, 16);
#pragma unroll
      for (int k = 0; k < N; ++k) __builtin_memcpy(x[k], x_row(k), 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i] = 0;
        if (i < 4)
#pragma unroll
          for (int k = 0; k < N; ++k) x[k][i] = 0;
      }
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        if (c + i >= a.hidden) break;
        if (a.type == LVQ_F32) r[i] = ((const uint32_t*)a.router)[row + c + i];
        else r[i >> 1] |= (uint32_t)((const uint16_t*)a.router)[row + c + i] << (16 * (i & 1));
#pragma unroll
        for (int k = 0; k < N; ++k) x[k][i >> 1] |= (uint32_t)x_row(k)[i] << (16 * (i & 1));
      }
    }
    double w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = (r[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
      const float v = a.type == LVQ_F32   ? __builtin_bit_cast(float, r[i])
                      : a.type == LVQ_F16 ? f16_to_f32(b)
                                          : __builtin_bit_cast(float, b << 16);
      w[i] = (double)v;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        acc[k] = __builtin_fma(w[i], (double)f16_to_f32((x[k][i >> 1] >> (16 * (i & 1))) & 0xFFFFu),
                               acc[k]);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const double s = wave_sum64_lane63(acc[k]);
    if ((threadIdx.x & 63) == 63) red[threadIdx.x >> 6][k] = s;
  }
  __syncthreads();
  if ((int)threadIdx.x < n) {
    const int k = threadIdx.x;
    double l = red[0][k];
    for (int w = 1; w < (int)blockDim.x / kWave; ++w) l += red[w][k];
    float* to = a.logits + (size_t)(t0 + k) * a.experts + e;
    *to = (float)l;
    to[(size_t)a.tokens * a.experts] = (float)(l - (double)(float)l);
  }
}

// ---------------------------------------------------------------- the choice

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  const uint32_t m = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
  return v > m ? v : m;
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = dpp_umax<0xB1>(v);
  v = dpp_umax<0x4E>(v);
  v = dpp_umax<0x141>(v);
  v = dpp_umax<0x140>(v);
  auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = p[0] > p[1] ? p[0] : p[1];
  auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return q[0] > q[1] ? q[0] : q[1];
}

// Integers of the floats' order, above 1 for all but NaN.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

// The top of a token's logits, by a wave: expert j goes to lane j's *id and *weight.
// Values are compared as integers of the same order, equal ones by their rests and then by their
// index.  A NaN is below everything, and makes the token's weights NaN.
// S: values per lane.
template <int S>
__device__ __forceinline__ void choose(const float* logits, const float* rests, int experts, int top,
                                       bool renormalize, int lane, int* id, float* weight) {
  float v[S];
  uint32_t key[S];
  bool nan = false;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = s * kWave + lane;
    v[s] = e < experts ? logits[e] + 0.f : -__builtin_inff();  // + 0: no negative zero
    key[s] = e >= experts ? 0u : v[s] != v[s] ? 1u : order_of(v[s]);
    nan |= v[s] != v[s];
  }
  nan = __any(nan);
  float best = 0.f, total = 0.f, mine = -__builtin_inff();
  int chosen = 0;
  for (int j = 0; j < top; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int s = 1; s < S; ++s) m = m > key[s] ? m : key[s];
    m = wave_umax(m);
    int e = 0, equal = 0;
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
      const uint64_t who = __ballot(key[s] == m);
      if (who) e = s * kWave + __builtin_ctzll(who);
      equal += __builtin_popcountll(who);
    }
    if (equal > 1) {
      // the rest of an infinity or a NaN is none
      uint32_t rest[S], most = 0;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        rest[s] = 0;
        if (key[s] == m) {
          const float r = rests[s * kWave + lane] + 0.f;
          rest[s] = order_of(r == r ? r : 0.f);
        }
        most = most > rest[s] ? most : rest[s];
      }
      most = wave_umax(most);
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        const uint64_t who = __ballot(key[s] == m && rest[s] == most);
        if (who) e = s * kWave + __builtin_ctzll(who);
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s * kWave + lane == e) key[s] = 0u;
    const float val = __builtin_bit_cast(float, (m >> 31) ? m & 0x7FFFFFFFu : ~m);
    if (j == 0) {
      best = val;
      if (!renormalize) {
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s)
          if (s * kWave < experts) sum += expf(v[s] - best);
        total = wave_sum(sum);
      }
    }
    if (lane == j) chosen = e, mine = val;
  }
  const float p = lane < top ? expf(mine - best) : 0.f;
  if (renormalize) total = wave_sum(p);
  *id = chosen;
  *weight = nan ? __builtin_nanf("") : p / total;
}

// A job: some tokens of one expert, up to four in the second launch and two in the third.  Its
// activations are rows first, first + 1, ... of the workspace: the pairs (token, chosen
// expert) sorted by expert, then by token.
struct __attribute__((aligned(8))) Job {
  uint16_t expert, first;
  uint16_t tokens;  // four bits each
  uint16_t count;
};
// What the second launch leaves for the third.
struct JobList {
  int n, pad[3];
  Job job[kMaxPairs];
  float weight[kMaxPairs];  // of a row of activations
};
struct JobSpace {
  uint16_t mask[kMaxExperts];   // tokens that chose the expert
  uint16_t start[kMaxExperts];  // its first row
  uint32_t total[kMaxExperts / kWave];
  int n;
  Job job[kMaxPairs];
};

// From the masks (complete, but for a barrier) the jobs, and the third launch's (to `list`
// unless NULL).  Every thread of the workgroup, at least kMaxExperts of them, calls.
__device__ __forceinline__ void make_jobs(JobSpace& j, JobList* list) {
  __syncthreads();
  const int e = threadIdx.x, lane = e & (kWave - 1), wv = e / kWave;
  uint32_t m = 0, sum = 0, own = 0;
  if (e < kMaxExperts) {
    m = j.mask[e];
    const uint32_t c = __builtin_popcount(m);
    own = sum = c | ((c + 3) / 4) << 10 | ((c + 1) / 2) << 20;  // rows, jobs of four, of two
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const uint32_t o = __shfl_up(sum, d, kWave);
      if (lane >= d) sum += o;
    }
    if (lane == kWave - 1) j.total[wv] = sum;
  }
  __syncthreads();
  if (e < kMaxExperts) {
    uint32_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kMaxExperts / kWave; ++w) {
      base += w < wv ? j.total[w] : 0;
      all += j.total[w];
    }
    base += sum - own;
    int row = base & 1023, at = base >> 10 & 1023, at2 = base >> 20;
    j.start[e] = (uint16_t)row;
    for (int left = own & 1023; left > 0; left -= 4, row += 4) {
      const int n = left < 4 ? left : 4;
      uint32_t t = 0;
      for (int b = 0; b < n; ++b) {
        t |= (uint32_t)__builtin_ctz(m) << (4 * b);
        m &= m - 1;
      }
      j.job[at++] = Job{(uint16_t)e, (uint16_t)row, (uint16_t)t, (uint16_t)n};
      if (list) {
        list->job[at2++] = Job{(uint16_t)e, (uint16_t)row, (uint16_t)t, (uint16_t)(n < 2 ? n : 2)};
        if (n > 2)
          list->job[at2++] =
              Job{(uint16_t)e, (uint16_t)(row + 2), (uint16_t)(t >> 8), (uint16_t)(n - 2)};
      }
    }
    if (e == 0) {
      j.n = (int)(all >> 10 & 1023);
      if (list) list->n = (int)(all >> 20);
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- gate and up

struct GateArgs {
  const uint8_t* codes;
  const uint16_t* scale;
  const uint16_t* zero;
  const uint16_t* x;
  const float* logits;
  JobList* jobs;
  int32_t* ids_out;  // may be NULL
  float* weights_out;
  uint16_t* act;     // [pairs][pitch] rounded values, then as many rests
  int hidden, inner, wgs;
  uint16_t tokens, experts, top;
  uint8_t gshift, renormalize, waves;
};
static_assert(sizeof(GateArgs) < 128, "launches of 128 bytes and more are slower");

// LDS of x: a token's row of steps, each four words of 16 units; 32 bytes more than they
// are long, so that four tokens' pieces lie in different banks.
__host__ __device__ inline int x_row_bytes(int steps) { return steps * 1024 + 32; }
inline size_t gate_lds_bytes(int tokens, int steps) {
  return (size_t)tokens * (x_row_bytes(steps) + steps * 64);
}

// Activations in the workspace: a row of whole steps, each as four words of 16 units, so that a
// load of one word of all units is of adjacent bytes; the eight values of a word in the
// order of the operands' pairs (the bits of their number reversed).
__host__ __device__ inline int act_pitch(int inner) { return (inner + 511) / 512 * 512; }
__device__ __forceinline__ int act_place(int c) {
  return (c & ~511) + (c >> 3 & 3) * 128 + (c >> 5 & 15) * 8 +
         ((c & 1) << 2 | (c & 2) | (c >> 2 & 1));
}

// Four steps of codes of a gate and an up quad; scales (low) and zeros of their groups.
template <int NS>
struct GateChunk {
  u32x4_t w[2][4];
  uint16_t s[2][NS], z[2][NS];
};

template <int NS, bool Z>
__global__ void __launch_bounds__(kGateWaves* kWave) moe_gate_kernel(GateArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ JobSpace jobs;
  const int nunits = (a.hidden + 31) / 32, steps = (nunits + 15) / 16;
  const int groups = ((nunits - 1) >> a.gshift) + 1;
  const int row_x = x_row_bytes(steps);
  uint8_t* xs = smem;
  float* sums = (float*)(smem + a.tokens * row_x);
  const int lane = threadIdx.x & (kWave - 1), ul = lane >> 2, r4 = lane & 3;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int nw = a.waves;

  // 1. the choice, a token per wave
  if (a.tokens > 1)
    for (int e = threadIdx.x; e < kMaxExperts; e += nw * kWave) jobs.mask[e] = 0;
  int id = 0;
  float weight = 0.f;
  const bool chooses = wv < a.tokens;
  if (chooses) {
    const float* l = a.logits + (size_t)wv * a.experts;
    const float* rests = l + (size_t)a.tokens * a.experts;
    // two values per lane where they hold all: eight cost 1.2 us more of the layer's (one token of
    // 2048 x 768, 8 chosen of 16, 64, 128: 14.6, 14.8, 15.0 us with two, 15.9, 16.0, 16.3 with
    // eight; of 256 and 512, with eight, 16.4 and 17.3)
    if (a.experts <= 2 * kWave) choose<2>(l, rests, a.experts, a.top, a.renormalize, lane, &id, &weight);
    else choose<kMaxExperts / kWave>(l, rests, a.experts, a.top, a.renormalize, lane, &id, &weight);
  }

  // 2. x into LDS, and minus the sums of its units, as the products start from them
  for (int i = wv; i < a.tokens * steps; i += nw) {
    const int t = i / steps, st = i - t * steps, c = (st * 64 + lane) * 8;
    const uint16_t* row = a.x + (size_t)t * a.hidden;
    u32x4_t v = {0, 0, 0, 0};
    if (c + 8 <= a.hidden) {
      __builtin_memcpy(&v, row + c, 16);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < a.hidden) v[k >> 1] |= (uint32_t)row[c + k] << (16 * (k & 1));
    }
    *(u32x4_t*)(xs + t * row_x + st * 1024 + r4 * 256 + ul * 16) = pair_order(v);
    constexpr uint32_t kOnes = 0x3C003C00u;
    float s = dot2(v.x, kOnes, dot2(v.y, kOnes, dot2(v.z, kOnes, dot2(v.w, kOnes, 0.f))));
    s = dpp_add<0x4E, 0xF>(dpp_add<0xB1, 0xF>(s));
    if (r4 == 0) sums[(t * steps + st) * 16 + ul] = s * ((Z ? -1.f : -8.f) * kMoeUnit);
  }
  const bool chose = chooses && lane < a.top;
  JobList* const list = blockIdx.x == 0 ? a.jobs : nullptr;
  int at = lane;
  if (a.tokens == 1) {  // a job per chosen expert, as they come
    const Job job = {(uint16_t)id, (uint16_t)lane, 0, 1};
    if (chose) jobs.job[lane] = job;
    if (threadIdx.x == 0) jobs.n = a.top;
    if (list && chose) list->job[lane] = job;
    if (list && threadIdx.x == 0) list->n = a.top;
    __syncthreads();
  } else {
    __syncthreads();
    // two experts may share a word: or-ed in whole words
    if (chose) atomicOr((uint32_t*)jobs.mask + id / 2, (uint32_t)1 << (wv + 16 * (id & 1)));
    make_jobs(jobs, list);
    if (chose) at = jobs.start[id] + __builtin_popcount(jobs.mask[id] & ((1u << wv) - 1));
  }
  if (list && chose) {
    list->weight[at] = weight;
    if (a.ids_out) a.ids_out[wv * a.top + lane] = id;
    if (a.weights_out) a.weights_out[wv * a.top + lane] = weight;
  }

  // 3. items: a job and four rows of the activation, whole rows of the weights
  // the padding of the last unit is written too, as zeros
  const int quads = (a.inner + 31) / 32 * 8;
  const int row_bytes = nunits * 16, chunks = (steps + 3) / 4;
  const int items = jobs.n * quads, stride = a.wgs * nw;
  const size_t lo = (size_t)a.tokens * a.top * act_pitch(a.inner);
  struct Cursor {
    int item, chunk;
  };
  Cursor ld = {(int)blockIdx.x * nw + wv, 0}, cu = ld;
  auto advance = [&](Cursor& c) {
    if (++c.chunk == chunks) c.chunk = 0, c.item += stride;
  };
  const int lane_off = r4 * row_bytes + ul * 16;
  GateChunk<NS> ring[2];
  auto load = [&](GateChunk<NS>& k) {
    // no branch around the loop's loads, so that each wait counts just those behind the one
    // it is for; past the last item they are of empty ranges
    const bool none = ld.item >= items;
    const int item = none ? 0 : ld.item;
    const int job = item / quads, quad = item - job * quads, t0 = ld.chunk * 4;
    const size_t e = __builtin_amdgcn_readfirstlane(jobs.job[job].expert);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = quad * 4 + (h ? a.inner : 0), left = 2 * a.inner - row;
      const int rows = none || left < 0 ? 0 : left < 4 ? left : 4;
      const size_t first = e * 2 * a.inner + (rows ? row : 0);
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const int t = t0 + n * (4 / NS);
        const int g = ((t * 16) >> a.gshift) + ul;
        const int off = ((r4 * groups + g) * 2) | ((groups - 1 - g) & (int)0x80000000);
        const uint32_t bytes = t < steps ? (uint32_t)(rows * groups) * 2 : 0;
        k.s[h][n] = __builtin_amdgcn_raw_buffer_load_b16(q4_rsrc(a.scale + first * groups, bytes),
                                                         off, 0, 0);
        if constexpr (Z)
          k.z[h][n] = __builtin_amdgcn_raw_buffer_load_b16(q4_rsrc(a.zero + first * groups, bytes),
                                                           off, 0, 0);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = quad * 4 + (h ? a.inner : 0), left = 2 * a.inner - row;
      const int rows = none || left < 0 ? 0 : left < 4 ? left : 4;
      const size_t first = e * 2 * a.inner + (rows ? row : 0);
      // offsets in the base and the lanes, as in the down product: the range then holds whether or
      // not a scalar offset counts in its check
      const uint8_t* base = a.codes + first * row_bytes + t0 * 256;
      const uint32_t bytes = rows ? rows * row_bytes - t0 * 256 : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        k.w[h][i] = __builtin_bit_cast(
            u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(q4_rsrc(base, t0 + i < steps ? bytes : 0),
                                                           lane_off + i * 256, 0, 2));
    }
    advance(ld);
  };
  float acc[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[h][b] = 0.f;
  const int from = (((ul >> a.gshift) << 2) | r4) << 2, from_step = (16 >> a.gshift) << 4;
  auto consume = [&](const GateChunk<NS>& k) {
    if (cu.item >= items) return;
    const int job = cu.item / quads, quad = cu.item - job * quads, t0 = cu.chunk * 4;
    const Job jb = jobs.job[job];
    const int nb = __builtin_amdgcn_readfirstlane(jb.count);
    const int first = __builtin_amdgcn_readfirstlane(jb.first);
    const int tokens = __builtin_amdgcn_readfirstlane(jb.tokens);
    auto token = [&](int b) { return tokens >> (4 * b) & 15; };  // 0 past the last
    const uint8_t* xl = xs + token(r4) * row_x + ul * 16 + t0 * 1024;
    const float* sl[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) sl[b] = sums + (token(b) * steps + t0) * 16 + ul;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t0 + i >= steps) break;
      constexpr int SPL = 4 / NS;
      uint32_t sz[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sz[h] = (uint32_t)k.s[h][i / SPL] | (Z ? (uint32_t)k.z[h][i / SPL] << 16 : 0x48000000u);
        if constexpr (NS < 4)
          sz[h] = (uint32_t)__builtin_amdgcn_ds_bpermute(from + (i % SPL) * from_step, (int)sz[h]);
      }
      float sx[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) sx[b] = sl[b][i * 16];
      float4_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 4; ++b) c[h][b] = Z ? f16_to_f32(sz[h] >> 16) * sx[b] : sx[b];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const u32x4_t x = *(const u32x4_t*)(xl + i * 1024 + w * 256);
        constexpr uint32_t m = 0x03C003C0u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t q = k.w[h][i][w];
          c[h] = __builtin_amdgcn_mfma_f32_4x4x4f16(
              __builtin_bit_cast(half4_t, u32x2_t{x.x, x.y}),
              __builtin_bit_cast(half4_t, u32x2_t{(q << 6) & m, (q >> 2) & m}), c[h], 0, 0, 0);
          c[h] = __builtin_amdgcn_mfma_f32_4x4x4f16(
              __builtin_bit_cast(half4_t, u32x2_t{x.z, x.w}),
              __builtin_bit_cast(half4_t, u32x2_t{(q << 2) & m, (q >> 6) & m}), c[h], 0, 0, 0);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s = f16_to_f32(sz[h]);
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[h][b] = __builtin_fmaf(s, c[h][b], acc[h][b]);
      }
    }
    advance(cu);
    if (cu.chunk) return;
    // the rows' end: sums over the units, the activation in lane 4 b + i of token b, row i
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b < nb) {
        const float gb = sum_blocks(acc[0][b]), ub = sum_blocks(acc[1][b]);
        g = ul == b ? gb : g, u = ul == b ? ub : u;
      }
      acc[0][b] = acc[1][b] = 0.f;
    }
    if (ul < nb) {
      g *= 1.f / kMoeUnit, u *= 1.f / kMoeUnit;
      // a quarter of 1 + e^-g is inverted: the hardware's 1/v is 0 where it would be subnormal
      const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
      float v = g * 0.25f * __builtin_amdgcn_rcpf(__builtin_fmaf(e, 0.25f, 0.25f)) * u;
      const int row = quad * 4 + r4;
      if (row >= a.inner) v = 0.f;
      asm("" : "+v"(v));  // one value for both: not multiplied and rounded at once for either
      const _Float16 hi = (_Float16)v, rest = (_Float16)((v - (float)hi) * kRestUnit);
      const size_t to = (size_t)(first + ul) * act_pitch(a.inner) + act_place(row);
      a.act[to] = __builtin_bit_cast(uint16_t, hi);
      a.act[lo + to] = __builtin_bit_cast(uint16_t, rest);
    }
  };
  if (ld.item + (chunks > 1 ? 0 : stride) < items) {  // two at least
    load(ring[0]);
    load(ring[1]);
    while (ld.item < items) {
      consume(ring[0]);
      load(ring[0]);
      consume(ring[1]);
      load(ring[1]);
    }
  } else if (ld.item < items) {
    load(ring[0]);
  }
  consume(ring[0]);
  consume(ring[1]);
}

// ---------------------------------------------------------------- down

// Orders a wave's LDS accesses (its LDS instructions execute in order).
__device__ __forceinline__ void lds_in_order() {
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

struct DownArgs {
  const uint8_t* codes;
  const uint16_t* scale;
  const uint16_t* zero;
  const uint16_t* act;
  const JobList* jobs;
  float* y;
  int hidden, inner;
  uint16_t tokens, top;
  uint8_t gshift;
};
static_assert(sizeof(DownArgs) < 128, "launches of 128 bytes and more are slower");

// A workgroup: 8 rows, all jobs; their steps are dealt to its waves in equal parts.  A lane's
// four operand rows are the rounded values and the rests of two tokens, so that one
// product takes both.  Codes and activations are loaded as they lie, 64 lanes one behind the
// other, and reach their lanes through LDS: loaded by the lanes that multiply them,
// four neighbours each read another row, and such a load takes the cache four times as
// long (sixteen tokens, 2048x768: 31 us like that, 26 so).
constexpr int kDownWaves = 16, kDownQuads = 2;
// LDS: four rows of 16 units, rows 32 bytes further apart than they are long, so that the
// eight lanes that read at once (two units of four rows) lie in different banks
constexpr int kCodesRow = 256 + 32, kActRow = 1024 + 32;
constexpr int kDownLds = kDownQuads * 4 * kCodesRow + 4 * kActRow;

// NS: loads of scales per step (8 groups of 8 rows each).
template <int NS, bool Z>
__global__ void __launch_bounds__(kDownWaves* kWave) moe_down_kernel(DownArgs a) {
  constexpr int NQ = kDownQuads, R = 4 * NQ, W = kDownWaves, RING = 3;
  __shared__ float part[W][LVQ_MAX_MOE_TOKENS * R];
  __shared__ __attribute__((aligned(16))) uint8_t stage[W][kDownLds];
  const int lane = threadIdx.x & (kWave - 1), ul = lane >> 2, r4 = lane & 3;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const codes_lds = stage[wv];
  uint8_t* const act_lds = codes_lds + NQ * 4 * kCodesRow;
  const int pairs = a.tokens * a.top;
  for (int i = lane; i < a.tokens * R; i += kWave) part[wv][i] = 0.f;
  // the list into LDS: a load from memory in the loop would wait for all that are on their way
  __shared__ Job jobs[kMaxPairs];
  __shared__ float weights[kMaxPairs];
  const int n_jobs = a.jobs->n;
  if ((int)threadIdx.x < pairs) {
    jobs[threadIdx.x] = a.jobs->job[threadIdx.x];
    weights[threadIdx.x] = a.jobs->weight[threadIdx.x];
  }
  __syncthreads();
  auto job_at = [&](int i) {
    const uint64_t j = *(const uint64_t*)&jobs[i];
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)j);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(j >> 32));
    return __builtin_bit_cast(Job, (uint64_t)hi << 32 | lo);
  };

  const int nunits = (a.inner + 31) / 32, steps = (nunits + 15) / 16;
  const int groups = ((nunits - 1) >> a.gshift) + 1;
  const int pitch = act_pitch(a.inner), row_bytes = nunits * 16;
  const int all = n_jobs * steps, per = (all + W - 1) / W;
  const int f0 = wv * per < all ? wv * per : all, f1 = f0 + per < all ? f0 + per : all;
  const int row0 = blockIdx.x * R;
  const int rows = a.hidden - row0 < R ? a.hidden - row0 : R;

  struct Step {
    u32x4_t x[4];
    u32x4_t w[NQ];
    uint16_t s[NS], z[NS];
  };
  struct Cursor {
    int f, job, t;
  };
  auto start = [&](int f) { return Cursor{f, f / steps, f - f / steps * steps}; };
  auto next = [&](Cursor& c) {
    ++c.f;
    if (++c.t == steps) c.t = 0, ++c.job;
  };
  Cursor ld = start(f0), at = ld;
  // scales: lane (ul, r4) asks for row 4 (ul / 8) + r4 of the rows, group ul % 8 of the step's
  const int scale_off = (4 * (ul >> 3) + r4) * groups + (ul & 7);
  int code_off[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) code_off[q] = (4 * q + (lane >> 4)) * row_bytes + (lane & 15) * 16;
  const size_t rests = (size_t)pairs * pitch;
  // where the job of the next load begins
  const uint8_t* codes;
  size_t scales;
  const uint16_t* act;
  int count;
  auto enter = [&](int i) {
    const Job j = job_at(i);
    const size_t first = (size_t)j.expert * a.hidden + row0;
    codes = a.codes + first * row_bytes;
    scales = first * groups;
    act = a.act + (size_t)j.first * pitch, count = j.count;
  };
  if (f0 < f1) enter(ld.job);
  auto load = [&](Step& k) {
    // no branch around the loads, as in the gate's
    const bool past = ld.f >= f1;
    const uint32_t sb = past ? 0 : (uint32_t)(rows * groups) * 2;
    const int g0 = (ld.t * 16) >> a.gshift;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const int off = ((scale_off + g0 + n * 8) * 2) |
                      ((groups - 1 - g0 - n * 8 - (ul & 7)) & (int)0x80000000);
      k.s[n] = __builtin_amdgcn_raw_buffer_load_b16(q4_rsrc(a.scale + scales, sb), off, 0, 0);
      if constexpr (Z)
        k.z[n] = __builtin_amdgcn_raw_buffer_load_b16(q4_rsrc(a.zero + scales, sb), off, 0, 0);
    }
    // row i: token i / 2 of the job, the rounded values or the rests; a range of the step's 1024
    // bytes each, an empty one where there is no second token
    const int there = ld.t * 16 + (lane & 15) >= nunits ? 0x80000000 : lane * 16;
    const uint32_t one = past ? 0 : 1024, two = count > 1 ? one : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      k.x[i] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                       q4_rsrc(act + ld.t * 512 + (i >> 1) * pitch + (i & 1) * rests,
                               i < 2 ? one : two),
                       there, 0, 0));
    const auto range = q4_rsrc(codes + ld.t * 256, past ? 0 : rows * row_bytes - ld.t * 256);
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      k.w[q] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                               range, code_off[q], 0, 2));
    const int job = ld.job;
    next(ld);
    if (ld.job != job && ld.f < f1) enter(ld.job);
  };
  float acc[NQ][4];
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[q][b] = 0.f;
  const int rel = ul >> a.gshift;  // this lane's group of the step's
  auto consume = [&](const Step& k) {
    if (at.f >= f1) return;
    constexpr uint32_t kOne = 0x00400040u, m = 0x03C003C0u;
    const half4_t ones = __builtin_bit_cast(half4_t, u32x2_t{kOne, kOne});
    u32x4_t xo[4], wo[NQ];
    lds_in_order();
#pragma unroll
    for (int i = 0; i < 4; ++i) *(u32x4_t*)(act_lds + i * kActRow + lane * 16) = k.x[i];
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      *(u32x4_t*)(codes_lds + (4 * q + (lane >> 4)) * kCodesRow + (lane & 15) * 16) = k.w[q];
    lds_in_order();
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      wo[q] = *(const u32x4_t*)(codes_lds + (4 * q + r4) * kCodesRow + ul * 16);
#pragma unroll
    for (int w = 0; w < 4; ++w)
      xo[w] = *(const u32x4_t*)(act_lds + r4 * kActRow + w * 256 + ul * 16);
    // the sums of x and of each quad's products: chains of their own
    float4_t sum = {0, 0, 0, 0}, c[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) c[q] = float4_t{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const half4_t x0 = __builtin_bit_cast(half4_t, u32x2_t{xo[w].x, xo[w].y});
      const half4_t x1 = __builtin_bit_cast(half4_t, u32x2_t{xo[w].z, xo[w].w});
      sum = __builtin_amdgcn_mfma_f32_4x4x4f16(x0, ones, sum, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const uint32_t v = wo[q][w];
        c[q] = __builtin_amdgcn_mfma_f32_4x4x4f16(
            x0, __builtin_bit_cast(half4_t, u32x2_t{(v << 6) & m, (v >> 2) & m}), c[q], 0, 0, 0);
      }
      sum = __builtin_amdgcn_mfma_f32_4x4x4f16(x1, ones, sum, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const uint32_t v = wo[q][w];
        c[q] = __builtin_amdgcn_mfma_f32_4x4x4f16(
            x1, __builtin_bit_cast(half4_t, u32x2_t{(v << 2) & m, (v >> 6) & m}), c[q], 0, 0, 0);
      }
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      // from the lane that holds the scale: row r4 of quad q, group rel
      uint32_t sz = 0;
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const uint32_t both = (uint32_t)k.s[n] | (Z ? (uint32_t)k.z[n] << 16 : 0x48000000u);
        const uint32_t v = (uint32_t)__builtin_amdgcn_ds_bpermute(
            ((q * 8 + (rel & 7)) * 4 + r4) * 4, (int)both);
        sz = n == 0 || (rel >> 3) == n ? v : sz;
      }
      const float s = f16_to_f32(sz), z = f16_to_f32(sz >> 16);
#pragma unroll
      for (int b = 0; b < 4; ++b)
        acc[q][b] = __builtin_fmaf(s, __builtin_fmaf(-z, sum[b], c[q][b]), acc[q][b]);
    }
    const int job = at.job;
    next(at);
    if (at.f < f1 && at.t) return;
    const Job jb = job_at(job);
    const float weight = ul < jb.count ? weights[jb.first + ul] : 0.f;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      constexpr float back = 1.f / kRestUnit;
      const float v0 = sum_blocks(__builtin_fmaf(acc[q][1], back, acc[q][0]));
      const float v1 = jb.count > 1 ? sum_blocks(__builtin_fmaf(acc[q][3], back, acc[q][2])) : 0.f;
      if (ul < jb.count) {
        float* to = &part[wv][(jb.tokens >> (4 * ul) & 15) * R + 4 * q + r4];
        *to = __builtin_fmaf(weight, (ul ? v1 : v0) * (1.f / kMoeUnit), *to);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[q][b] = 0.f;
    }
  };
  Step ring[RING];
  // the loop is entered with a whole ring on its way, as every round of it leaves one: else its
  // first wait would be for everything
  if (f1 - f0 >= RING) {
#pragma unroll
    for (int d = 0; d < RING; ++d) load(ring[d]);
    while (ld.f < f1) {
#pragma unroll
      for (int d = 0; d < RING; ++d) {
        consume(ring[d]);
        load(ring[d]);
      }
    }
  } else {
#pragma unroll
    for (int d = 0; d < RING - 1; ++d)
      if (ld.f < f1) load(ring[d]);
  }
#pragma unroll
  for (int d = 0; d < RING; ++d) consume(ring[d]);
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * R; i += W * kWave) {
    const int t = i / R, r = row0 + i - t * R;
    float v = part[0][i];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][i];
    if (r < a.hidden) a.y[(size_t)t * a.hidden + r] = v;
  }
}

// ---------------------------------------------------------------- launch

struct MoeSpace {
  size_t logits, jobs, act, all;
};
inline MoeSpace moe_space(int tokens, int inner, int experts, int top) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  MoeSpace s;
  const size_t pairs = (size_t)tokens * top;
  s.logits = 0;
  s.jobs = up((size_t)tokens * experts * 8);
  s.act = s.jobs + up(sizeof(JobList));
  s.all = s.act + up(pairs * act_pitch(inner) * 4);
  return s;
}

inline bool moe_sizes_ok(int tokens, int hidden, int inner, int experts, int top) {
  return tokens >= 0 && tokens <= LVQ_MAX_MOE_TOKENS && hidden >= 1 && inner >= 1 &&
         hidden <= 65536 && inner <= 65536 && (long long)tokens * hidden <= 65536 &&
         experts >= 1 && experts <= kMaxExperts && top >= 1 && top <= LVQ_MAX_MOE_TOP &&
         top <= experts;
}

template <int NS, bool Z>
int launch_gate(const GateArgs& a, size_t lds, hipStream_t st) {
  hipLaunchKernelGGL((moe_gate_kernel<NS, Z>), dim3(a.wgs), dim3(a.waves * kWave), lds, st, a);
  return launch_status();
}
template <bool Z>
int launch_gate(const GateArgs& a, size_t lds, hipStream_t st) {
  return a.gshift == 0   ? launch_gate<4, Z>(a, lds, st)
         : a.gshift == 1 ? launch_gate<2, Z>(a, lds, st)
                         : launch_gate<1, Z>(a, lds, st);
}

template <int NS>
int launch_down(const DownArgs& a, hipStream_t st) {
  const int rows = 4 * kDownQuads;
  const dim3 grid((a.hidden + rows - 1) / rows), block(kDownWaves * kWave);
  if (a.zero) hipLaunchKernelGGL((moe_down_kernel<NS, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((moe_down_kernel<NS, false>), grid, block, 0, st, a);
  return launch_status();
}

struct MoeRange {
  const void* p;
  size_t n;
};

}  // namespace lvq

using namespace lvq;

extern "C" size_t q4_moe_workspace(int tokens, int hidden, int inner, int experts, int top) {
  return moe_sizes_ok(tokens, hidden, inner, experts, top)
             ? moe_space(tokens, inner, experts, top).all : 0;
}

extern "C" int q4_moe(const uint16_t* x, int tokens, int hidden, const void* router,
                      int router_type, int experts, int top, int renormalize,
                      const uint8_t* gu_codes, const uint16_t* gu_scale, const uint16_t* gu_zero,
                      int gu_group, const uint8_t* down_codes, const uint16_t* down_scale,
                      const uint16_t* down_zero, int down_group, int inner, float* y,
                      int32_t* ids_out, float* weights_out, void* workspace,
                      size_t workspace_bytes, void* stream) {
  const int gs = group_shift(gu_group), ds = group_shift(down_group);
  if (!moe_sizes_ok(tokens, hidden, inner, experts, top) || gs < 0 || ds < 0 ||
      (router_type != LVQ_F32 && router_type != LVQ_F16 && router_type != LVQ_BF16) ||
      renormalize < 0 || renormalize > 1)
    return LVQ_E_SHAPE;
  if (tokens == 0) return LVQ_OK;
  if (!x || !router || !gu_codes || !gu_scale || !down_codes || !down_scale || !y || !workspace)
    return LVQ_E_NULL;
  const void* all[] = {x, router, gu_codes, gu_scale, gu_zero, down_codes, down_scale, down_zero, y,
                       ids_out, weights_out, workspace};
  for (const void* p : all)
    if (!aligned16(p)) return LVQ_E_ALIGN;
  const MoeSpace sp = moe_space(tokens, inner, experts, top);
  if (workspace_bytes < sp.all) return LVQ_E_SHAPE;
  const size_t pairs = (size_t)tokens * top;
  const size_t gu_rows = (size_t)experts * 2 * inner, down_rows = (size_t)experts * hidden;
  const size_t gu_meta = gu_rows * group_count(hidden, gu_group) * 2;
  const size_t down_meta = down_rows * group_count(inner, down_group) * 2;
  const MoeRange in[8] = {{x, (size_t)tokens * hidden * 2},
                          {router, (size_t)experts * hidden * (router_type == LVQ_F32 ? 4 : 2)},
                          {gu_codes, gu_rows * units_of(hidden) * 16},
                          {gu_scale, gu_meta},
                          {gu_zero, gu_meta},
                          {down_codes, down_rows * units_of(inner) * 16},
                          {down_scale, down_meta},
                          {down_zero, down_meta}};
  const MoeRange made[4] = {{y, (size_t)tokens * hidden * 4},
                            {ids_out, pairs * 4},
                            {weights_out, pairs * 4},
                            {workspace, sp.all}};
  for (int i = 0; i < 4; ++i) {
    for (const MoeRange& r : in)
      if (ranges_overlap(made[i].p, made[i].n, r.p, r.n)) return LVQ_E_SHAPE;
    for (int j = i + 1; j < 4; ++j)
      if (ranges_overlap(made[i].p, made[i].n, made[j].p, made[j].n)) return LVQ_E_SHAPE;
  }
  const int steps = steps_of(hidden);
  const size_t lds = gate_lds_bytes(tokens, steps);
  if (lds + sizeof(JobSpace) > device_lds_bytes()) return LVQ_E_SHAPE;
  uint8_t* w = (uint8_t*)workspace;
  hipStream_t st = (hipStream_t)stream;
  RouterArgs r = {x, router, (float*)(w + sp.logits), tokens, hidden, experts, router_type};
  clear_hip_error();
  const int columns = (hidden + 8 * kWave - 1) / (8 * kWave);  // in waves
  const dim3 threads((columns < kRouterWaves ? columns : kRouterWaves) * kWave);
  if (tokens == 1) hipLaunchKernelGGL(moe_router_kernel<1>, dim3(experts), threads, 0, st, r);
  else hipLaunchKernelGGL(moe_router_kernel<4>, dim3(experts, (tokens + 3) / 4), threads, 0, st, r);
  int e = launch_status();
  if (e) return e;
  GateArgs g;
  g.codes = gu_codes, g.scale = gu_scale, g.zero = gu_zero, g.x = x;
  g.logits = r.logits, g.jobs = (JobList*)(w + sp.jobs);
  g.ids_out = ids_out, g.weights_out = weights_out, g.act = (uint16_t*)(w + sp.act);
  g.hidden = hidden, g.inner = inner;
  g.tokens = (uint16_t)tokens, g.experts = (uint16_t)experts, g.top = (uint16_t)top;
  g.gshift = (uint8_t)gs, g.renormalize = (uint8_t)renormalize;
  // at most a job per pair
  const long long items = (long long)pairs * units_of(inner) * 8;
  // a workgroup per CU, of as many waves as there are items for; the jobs of more than
  // one token take kMaxExperts threads to sort
  const int cus = device_cus(), least = tokens > 1 ? kMaxExperts / kWave : 1;
  const long long need = (items + cus - 1) / cus;
  const int waves = need > kGateWaves ? kGateWaves : need < least ? least : (int)need;
  g.waves = (uint8_t)(waves < tokens ? tokens : waves);
  const long long wgs = (items + g.waves - 1) / g.waves;
  g.wgs = wgs < cus ? (int)wgs : cus;
  e = gu_zero ? launch_gate<true>(g, lds, st) : launch_gate<false>(g, lds, st);
  if (e) return e;
  DownArgs d = {down_codes, down_scale, down_zero, g.act, g.jobs, y, hidden, inner,
                (uint16_t)tokens, (uint16_t)top, (uint8_t)ds};
  return ds == 0 ? launch_down<2>(d, st) : launch_down<1>(d, st);
}
