// gfx950 kernels of the loss operators of include/zero_loss.h: softmax cross
// entropy and top-K distillation over a vocabulary head, with the gradient.
//
// The order of one call:
//   scan      finds the rows that take part and numbers them (live positions)
//   pack      copies the live rows of hidden, padded and aligned; rows that
//             take no part are never read, so what they hold does not matter
//   logits    [live, piece] = hidden W^T in tiles; the forward reduces each
//             tile to softmax partials, the gradient turns it into g
//   dhidden   += g W,   dweight = g^T hidden    (gradient, per piece)
// The gradient makes the logits again: with the loss 8 operations for each token,
// entry and dimension, in place of 6. Keeping them instead would be 4 bytes a logit
// written and read again, the time of a product over some 1100 dimensions, and the
// memory that the pieces are there to avoid.
// Every product is one tiled kernel over 16-bit operands with fp32 sums. fp32
// values go through it as three bf16 parts, x = hi + mid + lo exactly: bf16 has
// fp32's exponents, so every value keeps its 24 bits whatever stands beside it. Six
// of the nine part products are summed, small ones first; the other three are
// together below 2^-23 of a product. (Two fp16 parts and three products take half the
// time, 1024 x 50257 x 768 with gradients 1.12 ms in place of 1.90, but fp16 has 40
// bits between its largest value and its smallest step: what is further below the
// largest of whatever shares a scale is lost, and probabilities are.)
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "zero_loss_launch.h"

namespace zloss {
namespace {

typedef uint16_t u16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// For the lambdas that the product is made of: they share its registers, and one
// that is called instead of inlined puts them all into memory.
#define INLINE __attribute__((always_inline))

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What the scan leaves for the kernels after it.
struct Head {
  int live;         // rows that take part
  int splits;       // runs that dhidden's sum over a piece of the vocabulary is cut into
  float scale;      // what g is held at
  float inv_scale;
};

// The power of two that brings the finite `top` to [2^to, 2^(to + 1)), within 2^+-100,
// and 1 for zero.
__device__ __forceinline__ int scale_exponent(float top, int to) {
  if (top == 0.0f) return 0;
  const int e = to - ilogbf(top);
  return e < -100 ? -100 : e > 100 ? 100 : e;
}

// Per live row, for the logits' gradient
//   g = a exp(z / temperature - lse) - c - hit [j = target]
//     = a2 2^(z log2(e) / temperature - base) - c - ..
// with base the lse over ln 2, rounded to sixteenths, and the rest of it in a2.
struct RowParam {
  float a2, base, c, hit;
  int target;       // global vocabulary index, or -1
  float a, lse;
  int pad;
};
static_assert(sizeof(RowParam) == 32, "the plan counts 32 bytes a row");

// The part products of fp32 operands: (left part, right part), small ones first.
constexpr int kParts = 3;
constexpr int kSegs = 6;
__device__ __forceinline__ int seg_a(int seg) { return 0x001021 >> 4 * seg & 3; }  // 1 2 0 1 0 0
__device__ __forceinline__ int seg_b(int seg) { return 0x010201 >> 4 * seg & 3; }  // 1 0 2 0 1 0

// ---- Values ---------------------------------------------------------------
__device__ __forceinline__ u16 bf16_bits(float x) { return __builtin_bit_cast(u16, (__bf16)x); }
__device__ __forceinline__ u16 f16_bits(float x) { return __builtin_bit_cast(u16, (_Float16)x); }
__device__ __forceinline__ float bf16_float(u16 b) {
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}
__device__ __forceinline__ float f16_float(u16 b) {
  return (float)__builtin_bit_cast(_Float16, b);
}

// x = p[0] + p[1] + p[2] in bf16 parts: 8 bits each, and the remainders' signs. An
// infinity or NaN is its first part alone (the remainder would be NaN); a finite value
// that would round to infinity has bf16's largest.
__device__ __forceinline__ void split3(float x, u16 p[kParts]) {
  p[0] = bf16_bits(x);
  const bool finite = __builtin_isfinite(x);
  p[0] -= finite && (p[0] & 0x7fff) == 0x7f80;
  const float r = finite ? x - bf16_float(p[0]) : 0.0f;
  p[1] = bf16_bits(r);
  p[2] = bf16_bits(r - bf16_float(p[1]));
}

template <int DT>
__device__ __forceinline__ float load_value(const void* p, int64_t i) {
  if constexpr (DT == kF32) return static_cast<const float*>(p)[i];
  const u16 b = static_cast<const u16*>(p)[i];
  return DT == kBF16 ? bf16_float(b) : f16_float(b);
}

__device__ __forceinline__ float load_any(const void* p, int64_t i, int dtype) {
  return dtype == kF32 ? load_value<kF32>(p, i)
                       : dtype == kBF16 ? load_value<kBF16>(p, i) : load_value<kF16>(p, i);
}

__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, int wide) {
  return wide ? static_cast<const int64_t*>(p)[i] : (int64_t) static_cast<const int32_t*>(p)[i];
}

template <int DT>
__device__ __forceinline__ void store_value(void* p, int64_t i, float x) {
  if constexpr (DT == kF32) static_cast<float*>(p)[i] = x;
  else static_cast<u16*>(p)[i] = DT == kBF16 ? bf16_bits(x) : f16_bits(x);
}

// Four values of a result to four consecutive elements; `wide`: the address suits
// one store (one store at any address is no faster: 64 x 50000 x 1001 in fp32 with
// gradients 620 us either way). Results, and g, are stored past the caches' own choice of
// what to keep (non-temporal): they are larger than the caches, and what they would push
// out, the weights and hidden states, is still wanted (40 tokens x 131072 x 2048 with
// gradients: 428 us in place of 487; 1000 x 32000 x 2048 in fp16: 511 in place of 529).
template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t i, f32x4 x, bool wide) {
  if (wide) {
    if constexpr (DT == kF32) {
      __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(static_cast<float*>(p) + i));
    } else {
      u16 b[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) b[r] = DT == kBF16 ? bf16_bits(x[r]) : f16_bits(x[r]);
      __builtin_nontemporal_store(
          u32x2{b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16},
          reinterpret_cast<u32x2*>(static_cast<u16*>(p) + i));
    }
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) store_value<DT>(p, i + r, x[r]);
  }
}

// exp of x in fp32: the product with log2(e) is rounded once, the rest is the
// hardware's exp2 (1 ulp).
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// The multiple of 1/16 next to x: exact in fp32 (as are differences of such), so
// that an exponent of two relative to it is rounded once, by its own size.
__device__ __forceinline__ float sixteenths(float x) { return rintf(x * 16.0f) * 0.0625f; }

// From here on fp32 has no sixteenths. A base may then be off by more than the exponents
// of two that are normal, and what is relative to it infinite: exponents are taken from
// the largest logit itself, or held to what a probability can have, and the base's own
// rounding, as large as the logits', is let go.
constexpr float kHugeBase = 0x1p20f;

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x = fmaxf(x, __shfl_xor(x, d));
  return x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

__host__ __device__ __forceinline__ int round_up_int(int x, int m) { return (x + m - 1) / m * m; }

// ---- Rows: which take part ------------------------------------------------
enum RowState { kEmpty = 0, kLive = 1, kBad = 2 };

__device__ __forceinline__ int target_state(const Call& c, int64_t t) {
  const int64_t y = load_index(c.target, t, c.index64);
  return y == c.ignore_index ? kEmpty : (y >= 0 && y < c.plan.vocab) ? kLive : kBad;
}

// Entries first, first + step, .. of a distillation row: 1 for one that counts, 2
// for one out of range, or'ed.
__device__ __forceinline__ int entry_states(const Call& c, int64_t t, int first, int step) {
  int seen = 0;
  for (int k = first; k < c.k; k += step) {
    const int64_t i = load_index(c.target, t * c.index_stride + k, c.index64);
    if (i >= c.plan.vocab) seen |= 2;
    if (i >= 0 && load_any(c.teacher, t * c.logit_stride + k, c.teacher_dtype) != -INFINITY)
      seen |= 1;
  }
  return seen;
}
__device__ __forceinline__ int state_of(int seen) {
  return seen & 2 ? kBad : seen & 1 ? kLive : kEmpty;
}

// The teacher's logit of entry k of row t; padding has -inf.
__device__ __forceinline__ float entry_logit(const Call& c, int64_t t, int k) {
  return load_index(c.target, t * c.index_stride + k, c.index64) < 0
             ? -INFINITY
             : load_any(c.teacher, t * c.logit_stride + k, c.teacher_dtype);
}

// Distillation: one wave a row.
__global__ void __launch_bounds__(256) classify_kernel(Call c, uint8_t* state) {
  const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  if (t >= c.plan.tokens) return;
  int seen = entry_states(c, t, threadIdx.x % 64, 64);
  seen = (__any(seen & 1) ? 1 : 0) | (__any(seen & 2) ? 2 : 0);
  if (threadIdx.x % 64 == 0) state[t] = (uint8_t)state_of(seen);
}

// The largest |g| a row can have, and the size of its pull on its target (short of
// the smoothing, which all rows share). A row whose g cannot be finite has no say in
// the scale that the others share.
struct Reach {
  float top, pull;
};
__device__ __forceinline__ Reach row_reach(const Call& c, int64_t t) {
  const float u = fabsf(c.upstream[t * c.upstream_stride]) * c.temperature;
  const float top = c.z_loss != 0.0f ? u * (1.0f + 2.0f * c.z_loss * fabsf(c.lse_in[t])) : u;
  return top < INFINITY ? Reach{top, u} : Reach{0.0f, 0.0f};
}

// The scale that g is held at. In fp16 the largest |g| a row can have comes to (2^13,
// 2^15], inside its range with 27 bits below it that are not subnormal; in bf16 (and
// fp32's parts) to (1/2, 2], so that no product overflows whose result does not; and of
// the factors that do so, the one that makes the largest row's pull on its target
// a power of two: with one upstream gradient for all rows, as a mean has, the -1
// of every row the model is unsure of is then exact, in place of all of them being
// rounded the same way.
__device__ __forceinline__ void set_scale(const Call& c, Reach r, float* scale, float* inv_scale) {
  const int e = scale_exponent(r.top, c.plan.dtype == kF16 ? 14 : 0);
  // pull (1 - smoothing) = part 2^q: dividing by the part, in [1, 2), leaves 2^q
  const float pull = r.pull * (1.0f - c.smoothing);
  const float part = pull > 0x1p-80f && pull < 0x1p80f ? scalbnf(pull, -ilogbf(pull)) : 1.0f;
  *scale = ldexpf(1.0f, e) / part;
  *inv_scale = ldexpf(part, -e);
}

// Row t's g = a exp(z - lse) - c - hit [j = target].
__device__ __forceinline__ RowParam row_param(const Call& c, int64_t t, float scale) {
  RowParam rp = {};
  const float u = c.upstream[t * c.upstream_stride] * scale;
  rp.lse = c.lse_in[t];
  if (c.k == 0) {
    rp.a = c.z_loss != 0.0f ? u * (1.0f + 2.0f * c.z_loss * rp.lse) : u;
    rp.c = u * c.smoothing / (float)c.plan.vocab;
    rp.hit = u * (1.0f - c.smoothing);
    rp.target = (int)load_index(c.target, t, c.index64);
  } else {
    rp.a = u * c.temperature;
    rp.target = -1;
  }
  const double l2 = rp.lse * 1.4426950408889634;
  rp.base = sixteenths((float)l2);
  rp.a2 = fabsf(rp.base) >= kHugeBase ? rp.a : (float)(rp.a * exp2(rp.base - l2));
  return rp;
}

// dhidden has few tiles, [live, dim], and a long sum, over the piece's vocabulary,
// which may be cut into runs. A tile takes its run's steps and, with the slab that is
// written and read again, about sixteen more (taking four made 1600 live rows x
// 65536 x 2048 4% slower, nothing faster). Few tokens: the number of runs with which the
// rounds of 512 tiles that the chip holds at once end soonest. Else the tiles are
// started as dweight's of the same launch end: `full` rounds of 256, and `rest` in one
// more; they are done at the first time at which the units that were free from the
// start of that round, and those that were from its end, have had time for them all.
// Lane l looks at l + 1 runs.
__device__ __forceinline__ int choose_splits(const Call& c, int live) {
  const Plan& p = c.plan;
  const bool few = p.tokens <= kFewTokens;
  const int lane = threadIdx.x % 64, s = lane + 1, bn = few ? 64 : 256;
  const int across = (int)((p.dimp + 255) / 256);
  const int tiles = (live + bn - 1) / bn * across;
  const int steps = ((int)(p.piece / 64) + s - 1) / s, each = steps + 16;
  int cost;
  if (few) {
    cost = (tiles * s + 511) / 512 * each;
  } else {
    const int w_tiles = c.dweight != nullptr ? (int)(p.piece / 256) * across : 0;
    const int w_each = (live + 63) / 64 + 4;
    const int full = w_tiles / 256, rest = w_tiles % 256;
    // k tiles on each early unit, and what the late ones manage in that time
    int k = max(1, tiles * s / 256);
    const auto done = [&](int t) {
      return (256 - rest) * (t / each) + rest * (max(0, t - w_each) / each);
    };
    int t = k * each;
    while (done(t) < tiles * s) t += min(each, rest > 0 ? w_each : each);
    cost = full * w_each + max(t, rest > 0 ? w_each : 0);
  }
  if (s > 1 && (tiles * s > p.acc_tiles || steps < 4)) cost = 0x7fffffff;
  int best = cost;
#pragma unroll
  for (int d = 32; d; d >>= 1) best = min(best, __shfl_xor(best, d));
  return __builtin_ctzll(__ballot(cost == best)) + 1;
}

// One block numbers the live rows in order.
__global__ void __launch_bounds__(1024) scan_kernel(Call c) {
  Head* head = reinterpret_cast<Head*>(c.ws + c.plan.o_head);
  int* rowmap = reinterpret_cast<int*>(c.ws + c.plan.o_rowmap);
  int* pos = reinterpret_cast<int*>(c.ws + c.plan.o_pos);
  const uint8_t* state = reinterpret_cast<const uint8_t*>(c.ws + c.plan.o_state);
  __shared__ int counts[16];
  __shared__ Reach reaches[16];
  const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  int base = 0;
  Reach reach = {0.0f, 0.0f};
  for (int64_t t0 = 0; t0 < c.plan.tokens; t0 += 1024) {
    const int64_t t = t0 + tid;
    int st = kEmpty;
    if (t < c.plan.tokens) st = c.k == 0 ? target_state(c, t) : state[t];
    const uint64_t votes = __ballot(st == kLive);
    if (lane == 0) counts[wave] = __popcll(votes);
    __syncthreads();
    int before = base, total = 0;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) before += counts[w];
      total += counts[w];
    }
    __syncthreads();
    if (t < c.plan.tokens) {
      if (st == kLive) {
        const int at = before + __popcll(votes & ((1ull << lane) - 1));
        rowmap[at] = (int)t;
        pos[t] = at;
        if (c.plan.grad) {
          const Reach r = row_reach(c, t);
          reach = {fmaxf(reach.top, r.top), fmaxf(reach.pull, r.pull)};
        }
      } else {
        pos[t] = st == kEmpty ? -1 : -2;
      }
    }
    base += total;
  }
  const int splits = c.plan.grad && wave == 0 ? choose_splits(c, base) : 1;
  reach = {wave_max(reach.top), wave_max(reach.pull)};
  if (lane == 0) reaches[wave] = reach;
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < 16; ++w)
      reach = {fmaxf(reach.top, reaches[w].top), fmaxf(reach.pull, reaches[w].pull)};
    head->live = base;
    head->splits = splits;
    set_scale(c, reach, &head->scale, &head->inv_scale);
  }
}

// ---- Packing --------------------------------------------------------------
// Eight elements from column k of a row, zero beyond `dim`, as 16-bit parts. Rows may
// start at any element: the memory takes 16-byte loads at any address (loads element
// by element where rows are not aligned to 16 bytes: 64 x 50000 x 1001 in fp32 with
// gradients 697 us in place of 620, the loss of 8 x 50000 x 1001 in bf16 79 in place of 65).
template <int DT>
__device__ __forceinline__ void pack8(const void* src, int64_t at, int k, int dim,
                                      u32x4 out[kParts]) {
  if constexpr (DT != kF32) {
    if (k + 8 <= dim) {
      __builtin_memcpy(&out[0], static_cast<const u16*>(src) + at + k, 16);
      return;
    }
    u16 b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = k + i < dim ? static_cast<const u16*>(src)[at + k + i] : 0;
    out[0] = *reinterpret_cast<const u32x4*>(b);
  } else {
    const float* x = static_cast<const float*>(src) + at + k;
    float v[8];
    if (k + 8 <= dim) {
      __builtin_memcpy(v, x, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k + i < dim ? x[i] : 0.0f;
    }
    u16 parts[kParts][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u16 p[kParts];
      split3(v[i], p);
#pragma unroll
      for (int s = 0; s < kParts; ++s) parts[s][i] = p[s];
    }
#pragma unroll
    for (int s = 0; s < kParts; ++s) out[s] = *reinterpret_cast<const u32x4*>(parts[s]);
  }
}

// The live rows of hidden, zero rows up to the next multiple of kRowPad; for the
// gradient the rows' parameters too.
template <int DT>
__global__ void __launch_bounds__(256) pack_hidden_kernel(Call c) {
  const Plan& p = c.plan;
  const Head* head = reinterpret_cast<const Head*>(c.ws + p.o_head);
  const int live = head->live;
  const int r = blockIdx.x;
  if (r >= round_up_int(live, (int)kRowPad)) return;
  u16* dst = reinterpret_cast<u16*>(c.ws + p.o_h) + (int64_t)r * p.dimp;
  const bool real = r < live;
  const int64_t t = real ? reinterpret_cast<const int*>(c.ws + p.o_rowmap)[r] : 0;
  const int64_t at = t * c.hidden_stride;
  if (p.grad && threadIdx.x == 0) {
    RowParam rp = {};
    rp.target = -1;
    if (real) rp = row_param(c, t, head->scale);
    reinterpret_cast<RowParam*>(c.ws + p.o_rowp)[r] = rp;
  }
  for (int k = threadIdx.x * 8; k < p.dimp; k += 256 * 8) {
    u32x4 v[kParts] = {};
    if (real) pack8<DT>(c.hidden, at, k, (int)p.dim, v);
    for (int s = 0; s < (DT == kF32 ? kParts : 1); ++s)
      *reinterpret_cast<u32x4*>(dst + s * p.rows * p.dimp + k) = v[s];
  }
}

// Up to kFewTokens tokens of a 16-bit type: what classify, scan, pack and row_param
// do, in one launch (each costs 3 to 4 us, of some 50 that a call takes). Every
// block numbers the rows for itself and packs its one; the first also writes down
// what later kernels read. Row r of the copy, and its columns from blockIdx.y on.
template <int DT>
__global__ void __launch_bounds__(256) few_rows_kernel(Call c) {
  const Plan& p = c.plan;
  const int tid = threadIdx.x, lane = tid % 64, tokens = (int)p.tokens;
  __shared__ int states[kFewTokens], rowmap[kFewTokens];
  __shared__ float scale;
  if (c.k == 0) {
    if (tid < tokens) states[tid] = target_state(c, tid);
  } else {  // four lanes a row
    int seen = tid / 4 < tokens ? entry_states(c, tid / 4, tid % 4, 4) : 0;
    seen |= __shfl_xor(seen, 1);
    seen |= __shfl_xor(seen, 2);
    if (tid % 4 == 0) states[tid / 4] = state_of(seen);
  }
  __syncthreads();
  const int st = lane < tokens ? states[lane] : kEmpty;
  const uint64_t votes = __ballot(st == kLive);
  const int live = __popcll(votes), at = __popcll(votes & ((1ull << lane) - 1));
  const bool first = blockIdx.x == 0 && blockIdx.y == 0;
  if (tid < 64) {
    if (st == kLive) rowmap[at] = lane;
    if (first) {
      Head* head = reinterpret_cast<Head*>(c.ws + p.o_head);
      if (st == kLive) reinterpret_cast<int*>(c.ws + p.o_rowmap)[at] = lane;
      if (lane < tokens)
        reinterpret_cast<int*>(c.ws + p.o_pos)[lane] = st == kLive ? at : st == kEmpty ? -1 : -2;
      const int splits = p.grad ? choose_splits(c, live) : 1;
      Reach r = {0.0f, 0.0f};
      if (p.grad && st == kLive) r = row_reach(c, lane);
      r = {wave_max(r.top), wave_max(r.pull)};
      if (lane == 0) {
        float inv_scale;
        set_scale(c, r, &scale, &inv_scale);
        *head = {live, splits, scale, inv_scale};
      }
    }
  }
  __syncthreads();
  if (first && p.grad && tid < kFewTokens) {
    RowParam rp = {};
    rp.target = -1;
    if (tid < live) rp = row_param(c, rowmap[tid], scale);
    reinterpret_cast<RowParam*>(c.ws + p.o_rowp)[tid] = rp;
  }
  const int r = blockIdx.x, k = ((int)blockIdx.y * 256 + tid) * 8;
  if (k >= p.dimp) return;
  u32x4 v[kParts] = {};
  if (r < live) pack8<DT>(c.hidden, rowmap[r] * c.hidden_stride, k, (int)p.dim, v);
  *reinterpret_cast<u32x4*>(reinterpret_cast<u16*>(c.ws + p.o_h) + (int64_t)r * p.dimp + k) = v[0];
}

// Vocabulary rows [v0, v0 + piece) of the weight, zero rows beyond the last.
template <int DT>
__global__ void __launch_bounds__(256) pack_weight_kernel(Call c, int64_t v0) {
  const Plan& p = c.plan;
  const int64_t r = blockIdx.x;
  u16* dst = reinterpret_cast<u16*>(c.ws + p.o_w) + r * p.dimp;
  const bool real = v0 + r < p.vocab;
  for (int k = threadIdx.x * 8; k < p.dimp; k += 256 * 8) {
    u32x4 v[kParts] = {};
    if (real) pack8<DT>(c.weight, (v0 + r) * c.weight_stride, k, (int)p.dim, v);
    for (int s = 0; s < (DT == kF32 ? kParts : 1); ++s)
      *reinterpret_cast<u32x4*>(dst + s * p.piece * p.dimp + k) = v[s];
  }
}

// ---- The product ----------------------------------------------------------
// out[n][m] = sum_k A[m][k] B[n][k]. An operand is stored either with its inner
// index contiguous (row r, step k at r*ld + k) or with its rows contiguous
// (k*ld + r, `T` for transposed).
struct Operand {
  const u16* p;
  int64_t plane;   // elements between the parts of fp32 operands
  int64_t ld;
  int rows;        // row indices beyond rows - 1 are read as the last (group of 8) there is
  int steps;       // likewise inner indices, where the other operand holds zeros
};

struct Product {
  Operand a, b;
  int m, n;        // extents (n: the most there can be, where live_n)
  int inner;       // inner extent, a multiple of 64 (the most there can be, where live_inner)
  bool live_n, live_inner;  // the extent is the live count, rounded up to 64 for the inner one
  bool split;      // the inner extent is cut into head->splits runs
  int segs;        // 1, or kSegs part products
  int beside;      // blocks ahead of the tiles', a multiple of 8, that do epi.beside()
  const Head* head;
};

// BM x BN tiles, inner steps of 64, one or two LDS stages that global memory is copied
// into directly while the other is multiplied. Waves hold 128 x (BN / 4 or 32)
// of the tile in matrix instructions 16x16x32.
//
// LDS holds a tile as it lies in memory, rows of 128 bytes (inner index
// contiguous) or 2 BM, 2 BN bytes (rows contiguous), in 16-byte groups whose place in
// their row is exchanged by a function of the row, so that the lanes of one read
// fall on different banks. The copy writes lane after lane, so the exchange is
// made in the addresses it reads from. A transposed tile is turned by the
// transposing LDS read, four inner steps of 16 rows a time.
//
// What bounds it. A 256 x 256 tile's step is 2048 cycles of matrix instructions on
// each SIMD and takes some 2650: with the logits of 8192 x 131072 x 4096 (6.0 ms, 1.46
// PFLOP/s) the matrix units are busy 77% of the time at 1.75 GHz, which is what the card's
// power allows at that load; the library's product of these sizes, without the softmax,
// has them busy 82% at 1.73 GHz (6.0 ms). At 768 inner dimensions a tile's start and its
// epilogue, which nothing overlaps, leave 49% at 2.13 GHz, 1.04 PFLOP/s.
// Measured against it and slower (each beside what it was then):
// four waves of 128 x 128 with the sums in accumulation registers (a third less LDS
// reading, but nobody to work while a wave waits; 27.7 ms in place of 26.6 for the
// whole of that case), a ring of five stages of 32 steps with a meeting each (27.1 in
// place of 26.1: pieces of 64 bytes cost the copies more), blocks that stay and copy
// their next tile during the epilogue (26.5 and 26.3: what the start costs is back in
// registers spilled and rounds that no longer even out), copies issued in one go
// instead of a few matrix instructions apart (27.6 and 26.2: they hold up the issue).
typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int BM, int BN, int STAGES>
struct Shape {
  static constexpr int kWaveN = BN == 256 ? 64 : 32;
  static constexpr int kWavesM = BM / 128;
  static constexpr int kWaves = kWavesM * (BN / kWaveN);
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kStageB = BM * 128;         // bytes before a stage's right operand
  static constexpr int kStage = (BM + BN) * 128;
  static constexpr int kLds = STAGES * kStage;
};

// The inner step that a narrow tile of the logits, from vocabulary row m on, starts at.
__device__ __forceinline__ int first_step(int m, int tile_rows, int steps) {
  return m / tile_rows * 5 % steps;
}

// Byte offsets, from the tile's corner (r0 < o.rows: a tile starts on a real row), that
// a lane copies from with its wave's `instr`-th instruction of 64 groups.
template <bool T, int R>
__device__ __forceinline__ uint32_t copy_offset(const Operand& o, int r0, int instr, int lane) {
  if constexpr (!T) {
    const int r = instr * 8 + lane / 8;
    const int group = (lane % 8) ^ (lane / 8);
    return (uint32_t)(min(r0 + r, o.rows - 1) - r0) * (uint32_t)(o.ld * 2) + group * 16;
  } else {
    constexpr int kGroups = R / 8;  // in an inner step's row
    const int k = instr * (64 / kGroups) + lane / kGroups;
    const int turn = (k & 3) | ((k >> 3) & 1) << 2;
    const int group = (lane % kGroups) ^ (turn << 1);
    return (uint32_t)k * (uint32_t)(o.ld * 2) +
           (uint32_t)(min(r0 + group * 8, o.rows - 8) - r0) * 2;
  }
}

// 16 bytes a lane from base + offset to LDS, lane after lane from `to` (both the
// same in the whole wave). The compiler does not see it as a load, and so does
// not hold up the transposing reads, which it cannot tell apart from the stage
// that is being written, until it has landed: the waits are written out below. It
// sets M0 itself (and may do so in the addition that forms `to`); the load needs an
// instruction's time after that.
__device__ __forceinline__ void copy_to_lds(const char* base, uint32_t offset, uint32_t to) {
  asm volatile(
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "{m0}"(to), "v"(offset), "s"(base)
      : "memory");
}

// The operand registers of one matrix instruction: 16 rows from `at`, inner
// steps 32 ks + lane / 16 * 8 + 0..7.
template <bool T, int R>
__device__ __forceinline__ u32x4 fragment(lds_char* tile, int at, int ks, int lane) {
  if constexpr (!T) {
    const int off = (at + lane % 16) * 128 + (((ks * 4 + lane / 16) ^ (lane & 7)) * 16);
    return *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(tile + off);
  } else {
    const int i = lane % 16, g = lane / 16;
    const int turn = (i / 4) | (g & 1) << 2;
    const int off = (ks * 32 + g * 8 + i / 4) * (R * 2) + (((at / 16) ^ turn) * 32) + (i % 4) * 8;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<lds_s16x4*>(tile + off));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<lds_s16x4*>(tile + off + 4 * (R * 2)));
    const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
    return u32x4{a[0], a[1], b[0], b[1]};
  }
}

template <int DT, bool TA, bool TB, int BM, int BN, int STAGES, class Epi>
__device__ __forceinline__ void product_block(const Product& g, Epi epi, int block,
                                              char* smem) {
  using S = Shape<BM, BN, STAGES>;
  constexpr int MI = 8, NJ = S::kWaveN / 16;
  constexpr int kCopyA = BM / 8 / S::kWaves, kCopyB = BN / 8 / S::kWaves;
  lds_char* lds = (lds_char*)smem;
  const uint32_t lds_at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);

  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int live = g.head->live;
  const int n_ext = g.live_n ? live : g.n;
  const int inner = g.live_inner ? round_up_int(live, 64) : g.inner;
  // Tiles are numbered in strips four columns wide, and each of the chip's eight
  // dies (blocks go to them in turn) gets a run of them, so that the tiles in
  // flight on a die share rows and columns in its cache.
  const int mt = (g.m + BM - 1) / BM, nt = (n_ext + BN - 1) / BN;
  const int splits = g.split ? g.head->splits : 1;
  const int total = mt * nt * splits, run = (total + 7) / 8;
  int id = block - g.beside;
  if (id < 0) return epi.beside((int64_t)block * S::kWaves + wave);
  if (id / 8 >= run) return;
  id = (id % 8) * run + id / 8;
  if (id >= total) return;
  const int split = id / (mt * nt);
  id -= split * mt * nt;
  const int strip = id / (4 * mt), wide = min(4, nt - strip * 4);
  id -= strip * 4 * mt;
  const int m0 = id / wide * BM, n0 = (strip * 4 + id % wide) * BN;

  const int chunk = round_up_int((inner + splits - 1) / splits, 64);
  const int k_lo = min(inner, split * chunk), k_hi = min(inner, k_lo + chunk);
  const int steps = (k_hi - k_lo) / 64, all = steps * g.segs;
  const int wm = wave % S::kWavesM * 128, wn = wave / S::kWavesM * S::kWaveN;

  uint32_t oa[kCopyA], ob[kCopyB];
#pragma unroll
  for (int i = 0; i < kCopyA; ++i)
    oa[i] = copy_offset<TA, BM>(g.a, m0, wave * kCopyA + i, lane);
#pragma unroll
  for (int i = 0; i < kCopyB; ++i)
    ob[i] = copy_offset<TB, BN>(g.b, n0, wave * kCopyB + i, lane);
  const auto corner = [&](const Operand& o, bool t, int r0, int part) INLINE {
    return reinterpret_cast<const char*>(o.p + part * o.plane +
                                         (t ? k_lo * o.ld + r0 : r0 * o.ld + k_lo));
  };
  const int64_t step_a = TA ? g.a.ld * 128 : 128, step_b = TB ? g.b.ld * 128 : 128;
  const char* pa = corner(g.a, TA, m0, g.segs > 1 ? seg_a(0) : 0);
  const char* pb = corner(g.b, TB, n0, g.segs > 1 ? seg_b(0) : 0);
  // Few tokens: what counts is the weight's way from memory. Its rows are a power of
  // two apart more often than not, and blocks that all read the same columns would
  // ask the same channels: each row of tiles starts at another step and comes round.
  constexpr bool kTurned = BN == 64 && !TA && !TB;
  const int turn = kTurned && steps > 0 ? first_step(m0, BM, steps) : 0;
  int seg = 0, at = turn;  // the next step to copy
  pa += turn * step_a;
  pb += turn * step_b;
  // Instruction i of a step's copies, A's first.
  const auto copy_part = [&](int stage, int i) INLINE {
    const uint32_t to = lds_at + stage * S::kStage;
    if (i < kCopyA) copy_to_lds(pa, oa[i], to + (wave * kCopyA + i) * 1024);
    else copy_to_lds(pb, ob[i - kCopyA], to + S::kStageB + (wave * kCopyB + i - kCopyA) * 1024);
  };
  const auto before_copy = [&]() INLINE {
    if (TA && k_lo + at * 64 + 64 > g.a.steps) {
      // the weight's last rows: there are no more, and the other operand holds zeros
#pragma unroll
      for (int i = 0; i < kCopyA; ++i) {
        const int k = (wave * kCopyA + i) * (512 / BM) + lane / (BM / 8);
        const int over = max(0, k_lo + at * 64 + k - (g.a.steps - 1));
        oa[i] = copy_offset<TA, BM>(g.a, m0, wave * kCopyA + i, lane) -
                (uint32_t)over * (uint32_t)(g.a.ld * 2);
      }
    }
  };
  const auto after_copy = [&]() INLINE {
    pa += step_a;
    pb += step_b;
    if (kTurned && ++at == steps) {
      at = 0;
      pa -= steps * step_a;
      pb -= steps * step_b;
    }
    if (kTurned ? at == turn : ++at == steps) {
      if (!kTurned) at = 0;
      if (++seg < g.segs) {
        pa = corner(g.a, TA, m0, seg_a(seg)) + turn * step_a;
        pb = corner(g.b, TB, n0, seg_b(seg)) + turn * step_b;
        if constexpr (TA) {
#pragma unroll
          for (int i = 0; i < kCopyA; ++i)
            oa[i] = copy_offset<TA, BM>(g.a, m0, wave * kCopyA + i, lane);
        }
      }
    }
  };
  const auto copy = [&](int stage) INLINE {
    before_copy();
#pragma unroll
    for (int i = 0; i < kCopyA + kCopyB; ++i) copy_part(stage, i);
    after_copy();
  };

  f32x4 acc[MI][NJ] = {};
  u32x4 fa0[MI], fb0[NJ], fa1[MI], fb1[NJ];
  // Operand q of a half step, in the order the matrix instructions want them.
  const auto read_part = [&](int stage, int ks, int q, u32x4 (&fa)[MI], u32x4 (&fb)[NJ]) INLINE {
    lds_char* ta = lds + stage * S::kStage;
    const int j = q == 0 ? 0 : q - 1;
    if (q == 1) fa[0] = fragment<TA, BM>(ta, wm, ks, lane);
    else if (q <= NJ) fb[j] = fragment<TB, BN>(ta + S::kStageB, wn + j * 16, ks, lane);
    else fa[q - NJ] = fragment<TA, BM>(ta, wm + (q - NJ) * 16, ks, lane);
  };
  // Multiplies one half step, row by row of the wave's tile, and between the rows
  // reads the next half's operands (read_stage >= 0) and copies the next free
  // stage (copy_stage >= 0): both are issued in the matrix instructions' shadow.
  const auto half = [&](u32x4 (&fa)[MI], u32x4 (&fb)[NJ], int read_stage, int ks,
                        u32x4 (&na)[MI], u32x4 (&nb)[NJ], auto copies, int copy_stage) INLINE {
    constexpr int kReads = MI + NJ, kFirst = MI - 2;  // the last two rows cover the latency
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = mfma<DT>(fa[i], fb[j], acc[i][j]);
      if (read_stage >= 0) {
#pragma unroll
        for (int q = i * kReads / kFirst; q < min(kReads, (i + 1) * kReads / kFirst); ++q)
          read_part(read_stage, ks, q, na, nb);
      }
      if constexpr (decltype(copies)::value) {
        constexpr int n = kCopyA + kCopyB;
#pragma unroll
        for (int q = i * n / MI; q < (i + 1) * n / MI; ++q) copy_part(copy_stage, q);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using Yes = std::true_type;
  using No = std::false_type;
  // A stage's copies have landed, and every wave has read all of the other stage.
  const auto meet = [&]() INLINE {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
  };
  if (all > 0 && n0 + wn >= n_ext) {
    // no column of this wave's is real: it copies its share and keeps step
    copy(0);
    meet();
    if (all > 1) copy(1);
    for (int it = 0; it + 1 < all; ++it) {
      meet();
      if (it + 2 < all) copy(it & 1);
    }
    if constexpr (Epi::kTurns) meet();
  } else if (all > 0) {
    // Each half step's operands are read while the half before is multiplied, and
    // the block meets between them: there the second half is in registers, so the
    // stage may be copied over, and the matrix units have work on both sides.
    copy(0);
    meet();
    if (all > 1) copy(1);
#pragma unroll
    for (int q = 0; q < MI + NJ; ++q) read_part(0, 0, q, fa0, fb0);
    int it = 0;
    for (; it + 2 < all; ++it) {
      half(fa0, fb0, it & 1, 1, fa1, fb1, No{}, 0);
      meet();
      before_copy();
      half(fa1, fb1, (it + 1) & 1, 0, fa0, fb0, Yes{}, it & 1);
      after_copy();
    }
    if (it + 1 < all) {
      half(fa0, fb0, it & 1, 1, fa1, fb1, No{}, 0);
      meet();
      half(fa1, fb1, (it + 1) & 1, 0, fa0, fb0, No{}, 0);
      ++it;
    }
    half(fa0, fb0, it & 1, 1, fa1, fb1, No{}, 0);
    half(fa1, fb1, -1, 0, fa0, fb0, No{}, 0);
    if constexpr (Epi::kTurns) meet();
  }
  epi.template tile<MI, NJ>(m0 + wm, n0 + wn, n_ext, split, acc,
                            lds + wave * 4096);
}

template <int DT, bool TA, bool TB, int BM, int BN, int STAGES, class Epi>
__global__ void __launch_bounds__((Shape<BM, BN, STAGES>::kThreads), 2)
    product_kernel(Product g, Epi epi) {
  __shared__ __attribute__((aligned(1024))) char smem[Shape<BM, BN, STAGES>::kLds];
  product_block<DT, TA, TB, BM, BN, STAGES, Epi>(g, epi, (int)blockIdx.x, smem);
}

// ---- The targets' logits ----------------------------------------------------
// The targets' logits, by the same matrix instructions in the same order as the
// tiles', so that they are the same bits as the ones in the softmax's sum: in a
// loss near zero the two have to cancel. One wave has 16 (row, entry) pairs, one
// per lane % 16: sixteen live rows with their one target each, or sixteen
// entries of one row. It multiplies their 16 weight rows with their 16 hidden
// rows and keeps the diagonal. Pairs outside the piece are left for theirs.
template <int DT>
struct Gather {
  Call c;
  const u16* w;     // the piece's weights
  int64_t ldw, v0;
  int real;
  // Cross entropy takes few of the sixteen: the rows' first touch of a far page is
  // what takes time, and more waves wait for more of them at once.
  static constexpr int kRowsWave = 4;
  __host__ __device__ int64_t waves() const {
    return c.k == 0 ? (c.plan.tokens + kRowsWave - 1) / kRowsWave
                    : c.plan.tokens * ((c.k + 15) / 16);
  }
  __device__ __forceinline__ void wave(int64_t id) const;
};

template <int DT>
__device__ __forceinline__ void Gather<DT>::wave(int64_t id) const {
  const Plan& p = c.plan;
  const int live = reinterpret_cast<const Head*>(c.ws + p.o_head)->live;
  const int K = c.k == 0 ? 1 : c.k, per_row = (K + 15) / 16;
  const int lane = threadIdx.x % 64, q = lane % 16;
  const int row = (int)(c.k == 0 ? id * kRowsWave + q : id / per_row);
  const int k = c.k == 0 ? 0 : (int)(id % per_row) * 16 + q;
  int64_t m = -1;  // the pair's row in the piece
  int64_t t = 0;
  if (row < live && k < K && (c.k != 0 || q < kRowsWave)) {
    t = reinterpret_cast<const int*>(c.ws + p.o_rowmap)[row];
    m = load_index(c.target, c.k == 0 ? t : t * c.index_stride + k, c.index64);
    m = m < 0 ? -1 : m - v0;  // padding has no weight row
  }
  const bool mine = m >= 0 && m < real;
  if (!__any(mine)) return;
  const u16* h = reinterpret_cast<const u16*>(c.ws + p.o_h) +
                 (int64_t)min(row, live - 1) * p.dimp + lane / 16 * 8;
  const u16* a = w + (mine ? m : 0) * ldw + lane / 16 * 8;
  // the narrow tiles' order of steps, each pair in that of its own weight row
  const int turn = p.tile_n == 64 && mine ? first_step((int)m, p.tile_m, (int)p.dimp / 64) * 64 : 0;
  f32x4 acc = {};
  for (int seg = 0; seg < (DT == kF32 ? kSegs : 1); ++seg) {
    const u16* pa = a + (DT == kF32 ? seg_a(seg) * p.piece * p.dimp : 0);
    const u16* pb = h + (DT == kF32 ? seg_b(seg) * p.rows * p.dimp : 0);
    constexpr int kDeep = 8;  // pairs of loads on their way at a time
    for (int k0 = 0; k0 < p.dimp; k0 += kDeep * 32) {
      u32x4 va[kDeep], vb[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        int k = min(k0 + i * 32, (int)p.dimp - 32) + turn;
        k -= k >= p.dimp ? (int)p.dimp : 0;
        va[i] = *reinterpret_cast<const u32x4*>(pa + k);
        vb[i] = *reinterpret_cast<const u32x4*>(pb + k);
      }
#pragma unroll
      for (int i = 0; i < kDeep; ++i)
        if (k0 + i * 32 < p.dimp) acc = mfma<DT>(va[i], vb[i], acc);
    }
  }
  // lane l holds rows l / 16 * 4 + 0..3 of column l % 16
  if (mine && q / 4 == lane / 16) {
    const float sum = q % 4 == 0 ? acc[0] : q % 4 == 1 ? acc[1] : q % 4 == 2 ? acc[2] : acc[3];
    (c.k == 0 ? reinterpret_cast<float*>(c.ws + p.o_entry) : c.logit)[t * K + k] = sum;
  }
}

template <int DT>
__global__ void __launch_bounds__(256) gather_kernel(Gather<DT> g) {
  const int64_t waves = g.waves();
  for (int64_t id = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; id < waves;
       id += (int64_t)gridDim.x * 4)
    g.wave(id);
}

// ---- What happens to a tile -------------------------------------------------
// A wave holds MI x NJ squares of 16 x 16: column n0 + 16 j + lane % 16, rows
// m0 + 16 i + lane / 16 * 4 + 0..3.

// Sixteen columns of 128 results, four 16-bit values in a register pair (`part`,
// one for each square), become rows of 256 bytes through 4 KB of LDS that are the
// wave's own once the stages are done with: then a store has 16 bytes a lane and four
// whole rows, in place of 8 bytes and sixteen pieces of 32. put(row, group, value) gets
// the rows' 16-byte groups. Groups are exchanged by their row, so that neither side meets
// a bank twice.
template <class Put>
__device__ __forceinline__ void turn_rows(lds_char* turn, const u32x2 (&part)[8], Put put) {
  const int lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
  typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
  typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<lds_u32x2*>(turn + r * 256 + ((i * 2 + g / 2) ^ r) * 16 + g % 2 * 8) =
        part[i];
  // (a wave's LDS instructions are carried out in their order: only the compiler is
  // to be told)
  asm volatile("" ::: "memory");
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = q * 4 + g;
    put(row, r, *reinterpret_cast<lds_u32x4*>(turn + row * 256 + (r ^ row) * 16));
  }
  asm volatile("" ::: "memory");
}

// Forward: the tile's rows m are vocabulary, its columns n live rows. Each wave
// leaves, of its stretch of the vocabulary, a base near its largest logit (as an
// exponent of two), the sum of the exponentials relative to it, and the sum of
// the logits.
template <int DT>
struct StatEpi {
  Gather<DT> gather;  // what the launch's first blocks do, where it has any for that
  float2* stat;
  float* sum;       // nullptr where nobody asks for it
  int64_t cols;     // partials per row
  float inv_temp;
  int m_base;       // vocabulary index of m = 0
  int vocab;
  static constexpr bool kTurns = false;
  __device__ __forceinline__ void beside(int64_t wave) const { gather.wave(wave); }
  template <int MI, int NJ>
  __device__ __forceinline__ void tile(int m0, int n0, int n_ext, int, f32x4 (&acc)[MI][NJ],
                                       lds_char*) {
    static_assert(MI * 16 == kStatRows, "one partial per wave");
    const int lane = threadIdx.x % 64;
    const int m_hi = vocab - m_base;
    if (m0 >= round_up_int(m_hi, (int)kStatRows) || n0 >= n_ext) return;
    const float f = inv_temp * kLog2e;
    const bool edge = m0 + (int)kStatRows > m_hi;  // some of it is beyond the vocabulary
    // These exponentials are the kernel's second cost after the products: a maximum,
    // one fused multiply-add, the power of two (four times an addition's time) and
    // the sum are 26 cycles a logit, 3 us a tile that takes 16 for 768 dimensions.
    // What only some tiles need is kept out of the others' way.
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      float top = -INFINITY, total = 0.0f, plain = 0.0f;
      if (sum != nullptr) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            plain += m0 + i * 16 + lane / 16 * 4 + r < m_hi ? acc[i][j][r] : 0.0f;
      }
      if (edge) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (m0 + i * 16 + lane / 16 * 4 + r >= m_hi) acc[i][j][r] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        top = fmaxf(fmaxf(top, acc[i][j][0]), acc[i][j][1]);
        top = fmaxf(fmaxf(top, acc[i][j][2]), acc[i][j][3]);
      }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float base = top == -INFINITY ? 0.0f : sixteenths(top * f);
      const bool huge = fabsf(base) >= kHugeBase;
      if (!__any(huge)) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            total += __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], f, -base));
      } else {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float x = acc[i][j][r];
            total += __builtin_amdgcn_exp2f(huge ? (x - top) * f : fmaf(x, f, -base));
          }
      }
      total += __shfl_xor(total, 16);
      total += __shfl_xor(total, 32);
      const int n = n0 + j * 16 + lane % 16;
      const int64_t at = n * cols + (m_base + m0) / kStatRows;
      if (sum != nullptr) {
        plain += __shfl_xor(plain, 16);
        plain += __shfl_xor(plain, 32);
        if (lane < 16 && n < n_ext) sum[at] = plain;
      }
      if (lane < 16 && n < n_ext) stat[at] = make_float2(base, total);
    }
  }
};

// Gradient: the same tile becomes g, [rows][ld] with the vocabulary
// contiguous. Rows beyond the live ones and columns beyond the vocabulary, up to
// the end of the last tile, hold zeros, so that the products over g need not
// know either.
template <int DT>
struct GradEpi {
  const RowParam* rows;
  u16* g;
  int64_t plane, ld;
  float inv_temp;
  int m_base, m_ext;   // first vocabulary index, how many of it are real
  bool shift;          // rows have a constant to take off (label smoothing)
  static constexpr bool kTurns = true;
  __device__ __forceinline__ void beside(int64_t) const {}
  template <int MI, int NJ>
  __device__ __forceinline__ void tile(int m0, int n0, int n_ext, int, f32x4 (&acc)[MI][NJ],
                                       lds_char* turn) {
    constexpr int kPlanes = DT == kF32 ? kParts : 1;
    const int lane = threadIdx.x % 64;
    const float f = inv_temp * kLog2e;
    const bool edge = m0 + MI * 16 > m_ext || n0 + NJ * 16 > n_ext;
    RowParam rps[NJ];  // all loads on their way before the first is waited for
#pragma unroll
    for (int j = 0; j < NJ; ++j) rps[j] = rows[n0 + j * 16 + lane % 16];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int n = n0 + j * 16 + lane % 16;
      const RowParam& rp = rps[j];
      const int at = rp.target - m_base - m0 - lane / 16 * 4;  // 16 i + r where it is this lane's
      const bool huge = fabsf(rp.base) >= kHugeBase;
      if (!__any(huge)) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][j][r] = rp.a2 * __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], f, -rp.base));
      } else {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float x = fmaf(acc[i][j][r], f, -rp.base);
            acc[i][j][r] = rp.a2 * __builtin_amdgcn_exp2f(huge && x > 0.0f ? 0.0f : x);
          }
      }
      if (shift) {
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][j] -= rp.c;
      }
      if (__any(at >= 0 && at < MI * 16 && (at & 15) < 4)) {  // one row's target in 128: rare
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][j][r] -= at == i * 16 + r ? rp.hit : 0.0f;
      }
      if (edge) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n >= n_ext || m0 + i * 16 + lane / 16 * 4 + r >= m_ext) acc[i][j][r] = 0.0f;
      }
      u32x2 packed[kPlanes][MI];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        u16 parts[kPlanes][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = acc[i][j][r];
          if constexpr (DT == kF32) {
            u16 p[kParts];
            split3(x, p);
            for (int s = 0; s < kParts; ++s) parts[s][r] = p[s];
          } else {
            parts[0][r] = DT == kBF16 ? bf16_bits(x) : f16_bits(x);
          }
        }
#pragma unroll
        for (int s = 0; s < kPlanes; ++s)
          packed[s][i] = u32x2{parts[s][0] | (uint32_t)parts[s][1] << 16,
                               parts[s][2] | (uint32_t)parts[s][3] << 16};
      }
#pragma unroll
      for (int s = 0; s < kPlanes; ++s)
        turn_rows(turn, packed[s], [&](int row, int group, u32x4 v) {
          __builtin_nontemporal_store(
              v, reinterpret_cast<u32x4*>(g + s * plane + (n0 + j * 16 + row) * ld + m0 +
                                          group * 8));
        });
    }
  }
};

// dhidden's sum over the vocabulary: fp32 [splits][live][ld], added to from the
// second piece on. Rows m are hidden's columns, columns n live rows.
struct SumEpi {
  float* acc_out;
  int64_t ld;
  int m_ext;
  bool add;
  static constexpr bool kTurns = false;
  __device__ __forceinline__ void beside(int64_t) const {}
  template <int MI, int NJ>
  __device__ __forceinline__ void tile(int m0, int n0, int n_ext, int split,
                                       f32x4 (&acc)[MI][NJ], lds_char*) {
    const int lane = threadIdx.x % 64;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int n = n0 + j * 16 + lane % 16;
      if (n >= n_ext) continue;
      float* to = acc_out + ((int64_t)split * n_ext + n) * ld + m0 + lane / 16 * 4;
      const int left = m_ext - m0 - lane / 16 * 4;
      if (add) {
        // eight loads at once: one after the other, each store's data would wait for its own
        f32x4 old[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i)
          old[i] = *reinterpret_cast<const f32x4*>(to + (i * 16 < left ? i * 16 : 0));
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][j] += old[i];
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
        if (i * 16 < left) *reinterpret_cast<f32x4*>(to + i * 16) = acc[i][j];
    }
  }
};

// dweight: rows m are hidden's columns, columns n the piece's vocabulary.
template <int DT>
struct WeightEpi {
  void* out;
  int64_t ld;
  int64_t v0;
  int m_ext;
  int wide;        // rows start at multiples of this many elements' size: 8, 4 or 1
  const Head* head;
  static constexpr bool kTurns = DT != kF32;
  __device__ __forceinline__ void beside(int64_t) const {}
  template <int MI, int NJ>
  __device__ __forceinline__ void tile(int m0, int n0, int n_ext, int, f32x4 (&acc)[MI][NJ],
                                       lds_char* turn) {
    const int lane = threadIdx.x % 64;
    const float s = head->inv_scale;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if constexpr (DT != kF32) {
        if (wide == 8) {
          u32x2 packed[MI];
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            const f32x4 x = acc[i][j] * s;
            u16 b[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) b[r] = DT == kBF16 ? bf16_bits(x[r]) : f16_bits(x[r]);
            packed[i] = u32x2{b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16};
          }
          turn_rows(turn, packed, [&](int row, int group, u32x4 v) {
            const int n = n0 + j * 16 + row, m = m0 + group * 8;
            if (n >= n_ext) return;
            u16* to = static_cast<u16*>(out) + (v0 + n) * ld + m;
            if (m + 8 <= m_ext) {
              __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(to));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (m + e < m_ext) to[e] = (u16)(v[e / 2] >> (16 * (e % 2)));
            }
          });
          continue;
        }
      }
      const int n = n0 + j * 16 + lane % 16;
      if (n >= n_ext) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int m = m0 + i * 16 + lane / 16 * 4;
        const f32x4 x = acc[i][j] * s;
        if (m + 4 <= m_ext) {
          store4<DT>(out, (v0 + n) * ld + m, x, wide >= 4);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (m + r < m_ext) store_value<DT>(out, (v0 + n) * ld + m + r, x[r]);
        }
      }
    }
  }
};

// Both products over a piece's g in one launch, dweight's tiles first: its last round
// of tiles seldom fills the chip, and dhidden's, whose size choose_splits() picks, go
// beside it. (4095 x 50257 x 768: two launches took 690 us, this one 600.)
template <int DT>
__global__ void __launch_bounds__(512, 2)
    gradients_kernel(Product w, WeightEpi<DT> we, int first, Product d, SumEpi de) {
  __shared__ __attribute__((aligned(1024))) char smem[Shape<256, 256, 2>::kLds];
  if ((int)blockIdx.x < first)
    product_block<DT, true, true, 256, 256, 2, WeightEpi<DT>>(w, we, (int)blockIdx.x, smem);
  else
    product_block<DT, true, false, 256, 256, 2, SumEpi>(d, de, (int)blockIdx.x - first, smem);
}

// ---- Rows: the losses -------------------------------------------------------
template <int N>
__device__ __forceinline__ float block_max(float x, float* s) {
  x = wave_max(x);
  __syncthreads();
  if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = x;
  __syncthreads();
  for (int w = 0; w < N; ++w) x = fmaxf(x, s[w]);
  return x;
}
template <int N>
__device__ __forceinline__ float block_sum(float x, float* s) {
  x = wave_sum(x);
  __syncthreads();
  if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = x;
  __syncthreads();
  x = 0.0f;
  for (int w = 0; w < N; ++w) x += s[w];
  return x;
}

// One block a token: joins the partials and writes the loss.
__global__ void __launch_bounds__(256) loss_kernel(Call c) {
  const Plan& p = c.plan;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  const int K = c.k == 0 ? 1 : c.k;
  __shared__ float red[4];
  __shared__ float ls[1024];
  const int at = reinterpret_cast<const int*>(c.ws + p.o_pos)[t];
  if (at < 0) {
    if (tid == 0) {
      c.loss[t] = at == -2 ? __builtin_nanf("") : 0.0f;
      c.lse[t] = 0.0f;
    }
    if (c.logit != nullptr)
      for (int k = tid; k < K; k += 256) c.logit[t * K + k] = 0.0f;
    return;
  }
  // base and sum s of 2^(z f - base) over the vocabulary, f = log2(e) / temperature
  const float2* stat = reinterpret_cast<const float2*>(c.ws + p.o_stat) + at * p.stat_cols;
  const int cols = (int)((p.vocab + kStatRows - 1) / kStatRows);
  float m = -INFINITY;
  for (int i = tid; i < cols; i += 256)
    if (stat[i].y > 0.0f) m = fmaxf(m, stat[i].x);
  m = block_max<4>(m, red);
  if (m == -INFINITY) m = 0.0f;
  float s = 0.0f, plain = 0.0f;
  for (int i = tid; i < cols; i += 256) {
    const float2 q = stat[i];
    s += q.y == 0.0f ? 0.0f : q.y * __builtin_amdgcn_exp2f(q.x - m);
  }
  s = block_sum<4>(s, red);
  if (c.smoothing != 0.0f) {
    const float* sum = reinterpret_cast<const float*>(c.ws + p.o_sum) + at * p.stat_cols;
    for (int i = tid; i < cols; i += 256) plain += sum[i];
    plain = block_sum<4>(plain, red);
  }
  const float* zs = (c.k == 0 ? reinterpret_cast<const float*>(c.ws + p.o_entry) : c.logit) + t * K;
  const float inv_temp = 1.0f / c.temperature, f = inv_temp * kLog2e;
  const float log2s = log2f(s), lse = (float)(((double)m + log2s) * 0.6931471805599453);
  // base - z f in one rounding: added to log2 s it is the loss in powers of two, and
  // exact where the target is the largest logit, since the sum has the same term.
  const auto behind = [m, f](float z) { return fmaf(-z, f, m); };
  if (c.k == 0) {
    if (tid == 0) {
      const float zy = zs[0];
      float loss = (behind(zy) + log2s) * kLn2;
      if (c.smoothing != 0.0f) loss += c.smoothing * (zy - plain / (float)p.vocab);
      if (c.z_loss != 0.0f) loss += c.z_loss * lse * lse;
      c.loss[t] = loss;
      c.lse[t] = lse;
    }
    return;
  }
  float top = -INFINITY;
  for (int k = tid; k < K; k += 256) {
    const float l = entry_logit(c, t, k);
    if (l == -INFINITY) c.logit[t * K + k] = 0.0f;
    ls[k] = l * inv_temp;
    top = fmaxf(top, ls[k]);
  }
  top = block_max<4>(top, red);
  float total = 0.0f;
  for (int k = tid; k < K; k += 256) total += exp_f(ls[k] - top);
  total = block_sum<4>(total, red);
  const float log_total = logf(total);
  float kl = 0.0f;
  for (int k = tid; k < K; k += 256) {
    const float lp = ls[k] - top - log_total;
    const float pk = exp_f(ls[k] - top) / total;
    if (ls[k] != -INFINITY) kl += pk * (lp + behind(zs[k]) * kLn2);
  }
  kl = block_sum<4>(kl, red);
  if (tid == 0) {
    c.loss[t] = c.temperature * c.temperature * (kl + log2s * kLn2);
    c.lse[t] = lse;
  }
}

// ---- Rows: the gradient -----------------------------------------------------
// Distillation: g at the teacher's entries that lie in the piece, written over
// what the tile left there: formed in one go from the saved logit, so that it
// too is rounded once. One wave a live row.
template <int DT>
__global__ void __launch_bounds__(64) entry_kernel(Call c, int64_t v0) {
  const Plan& p = c.plan;
  const int r = blockIdx.x, lane = threadIdx.x;
  if (r >= reinterpret_cast<const Head*>(c.ws + p.o_head)->live) return;
  __shared__ int idx[1024 + 8];
  __shared__ float pk[1024 + 8];
  if (lane < 8) {  // the search below goes by eights
    idx[c.k + lane] = -2;
    pk[c.k + lane] = 0.0f;
  }
  const int64_t t = reinterpret_cast<const int*>(c.ws + p.o_rowmap)[r];
  const RowParam rp = reinterpret_cast<const RowParam*>(c.ws + p.o_rowp)[r];
  const float inv_temp = 1.0f / c.temperature;
  float top = -INFINITY;
  for (int k = lane; k < c.k; k += 64) {
    const float l = entry_logit(c, t, k);
    idx[k] = l == -INFINITY ? -1 : (int)load_index(c.target, t * c.index_stride + k, c.index64);
    pk[k] = l * inv_temp;
    top = fmaxf(top, pk[k]);
  }
  top = wave_max(top);
  float total = 0.0f;
  for (int k = lane; k < c.k; k += 64) {
    const float e = exp_f(pk[k] - top);
    pk[k] = e;
    total += e;
  }
  total = wave_sum(total);
  __syncthreads();
  u16* g = reinterpret_cast<u16*>(c.ws + p.o_g) + (int64_t)r * p.piece;
  for (int k = lane; k < c.k; k += 64) {
    const int64_t m = idx[k] - v0;
    if (idx[k] < 0 || m < 0 || m >= p.piece) continue;
    const float z = c.logit_in[t * c.k + k] * inv_temp;
    const int own = idx[k];
    float same = 0.0f;
    for (int q = 0; q < c.k; q += 8)
#pragma unroll
      for (int e = 0; e < 8; ++e) same += idx[q + e] == own ? pk[q + e] : 0.0f;
    const float below = z - rp.lse;  // above only by rounding
    const float x = rp.a * (exp_f(below > 0.0f ? 0.0f : below) - same / total);
    if constexpr (DT == kF32) {
      u16 parts[kParts];
      split3(x, parts);
      for (int s = 0; s < kParts; ++s) g[s * p.rows * p.piece + m] = parts[s];
    } else {
      g[m] = DT == kBF16 ? bf16_bits(x) : f16_bits(x);
    }
  }
}

// Joins the slabs of dhidden's sum and writes every row, zeros where the row
// took no part. A wave has 256 columns of a row.
template <int DT>
__global__ void __launch_bounds__(64) dhidden_kernel(Call c, bool wide) {
  const Plan& p = c.plan;
  const int64_t t = blockIdx.x;
  const int at = reinterpret_cast<const int*>(c.ws + p.o_pos)[t];
  const Head* head = reinterpret_cast<const Head*>(c.ws + p.o_head);
  const int k = (int)blockIdx.y * 256 + threadIdx.x * 4;
  if (k >= p.dim) return;
  f32x4 x = {};
  if (at >= 0) {
    const float* acc = reinterpret_cast<const float*>(c.ws + p.o_acc) + (int64_t)at * p.dimp + k;
    const int splits = head->splits;
    const int64_t slab = (int64_t)head->live * p.dimp;
    for (int q = 0; q < splits; q += 8) {
      f32x4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = *reinterpret_cast<const f32x4*>(acc + min(q + i, splits - 1) * slab);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (q + i < splits) x += v[i];
    }
    x = x * head->inv_scale;
  }
  if (k + 4 <= p.dim) {
    store4<DT>(c.dhidden, t * c.dhidden_stride + k, x, wide);
  } else {
    for (int r = 0; r < 4 && k + r < p.dim; ++r)
      store_value<DT>(c.dhidden, t * c.dhidden_stride + k + r, x[r]);
  }
}

// ---- Launches -----------------------------------------------------------------
bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int64_t element(int dt) { return dt == kF32 ? 4 : 2; }

// Whether every row of a tensor starts at a multiple of `n` elements' size.
bool rows_aligned(const void* p, int64_t stride, int dt, int n) {
  return aligned(p, (uintptr_t)(n * element(dt))) && stride % n == 0;
}

template <int DT, bool TA, bool TB, int BM, int BN, int STAGES, class Epi>
void product_tiles(const Product& g, const Epi& epi, int64_t most_split, hipStream_t st) {
  int64_t total = (int64_t)((g.m + BM - 1) / BM) * ((g.n + BN - 1) / BN);
  if (g.split && total < most_split) total = most_split;
  const unsigned blocks = (unsigned)((total + 7) / 8 * 8 + g.beside);
  product_kernel<DT, TA, TB, BM, BN, STAGES, Epi>
      <<<blocks, Shape<BM, BN, STAGES>::kThreads, 0, st>>>(g, epi);
}

// The logits, in the plan's tiles.
template <int DT, class Epi>
void logits(const Plan& p, const Product& g, const Epi& epi, hipStream_t st) {
  if (p.tile_n == 256) product_tiles<DT, false, false, 256, 256, 2, Epi>(g, epi, 0, st);
  else if (p.tile_m == 256) product_tiles<DT, false, false, 256, 64, 2, Epi>(g, epi, 0, st);
  else product_tiles<DT, false, false, 128, 64, 2, Epi>(g, epi, 0, st);
}

template <int DT>
void rows_and_hidden(const Call& c, hipStream_t st) {
  const Plan& p = c.plan;
  if (DT != kF32 && p.tokens > 0 && p.tokens <= kFewTokens) {
    few_rows_kernel<DT><<<dim3(kFewTokens, (unsigned)((p.dimp + 2047) / 2048)), 256, 0, st>>>(
        c);
    return;
  }
  if (c.k > 0 && p.tokens > 0)
    classify_kernel<<<(unsigned)((p.tokens + 3) / 4), 256, 0, st>>>(
        c, reinterpret_cast<uint8_t*>(c.ws + p.o_state));
  scan_kernel<<<1, 1024, 0, st>>>(c);
  if (p.tokens > 0)
    pack_hidden_kernel<DT><<<(unsigned)p.rows, 256, 0, st>>>(c);
}

// The piece's weights as an operand source: packed, or where they are.
template <int DT>
const u16* piece_weight(const Call& c, int64_t v0, int64_t* ld, hipStream_t st) {
  const Plan& p = c.plan;
  if (!p.pack_w) {
    *ld = c.weight_stride;
    return static_cast<const u16*>(c.weight) + v0 * c.weight_stride;
  }
  pack_weight_kernel<DT><<<(unsigned)p.piece, 256, 0, st>>>(c, v0);
  *ld = p.dimp;
  return reinterpret_cast<const u16*>(c.ws + p.o_w);
}

template <int DT>
Product logits_product(const Call& c, const u16* w, int64_t ldw, int64_t real) {
  const Plan& p = c.plan;
  Product g{};
  g.a = {w, p.piece * p.dimp, ldw, (int)real, (int)p.dimp};
  g.b = {reinterpret_cast<const u16*>(c.ws + p.o_h), p.rows * p.dimp, p.dimp, (int)p.rows,
         (int)p.dimp};
  g.m = (int)real;
  g.n = (int)p.rows;
  g.inner = (int)p.dimp;
  g.live_n = true;
  g.segs = DT == kF32 ? kSegs : 1;
  g.head = reinterpret_cast<const Head*>(c.ws + p.o_head);
  return g;
}

template <int DT>
void loss_type(const Call& c, hipStream_t st) {
  const Plan& p = c.plan;
  rows_and_hidden<DT>(c, st);
  for (int64_t v0 = 0; v0 < p.vocab; v0 += p.piece) {
    int64_t ldw;
    const u16* w = piece_weight<DT>(c, v0, &ldw, st);
    const int64_t real = p.vocab - v0 < p.piece ? p.vocab - v0 : p.piece;
    const Gather<DT> gather{c, w, ldw, v0, (int)real};
    StatEpi<DT> epi{gather, reinterpret_cast<float2*>(c.ws + p.o_stat),
                    c.smoothing != 0.0f ? reinterpret_cast<float*>(c.ws + p.o_sum) : nullptr,
                    p.stat_cols, 1.0f / c.temperature, (int)v0, (int)p.vocab};
    Product g = logits_product<DT>(c, w, ldw, real);
    const int64_t blocks = (gather.waves() + 3) / 4, pairs = (gather.waves() + 1) / 2;
    // Few tokens: the gather's few waves, which wait for memory ten times over, go
    // beside the tiles (8 to 13 us less). More would take the tiles' room in LDS.
    if (p.tokens <= kFewTokens) g.beside = (int)(pairs + 7) / 8 * 8;
    logits<DT>(p, g, epi, st);
    if (p.tokens > kFewTokens)
      gather_kernel<DT><<<(unsigned)(blocks < (1 << 20) ? blocks : 1 << 20), 256, 0, st>>>(gather);
  }
  loss_kernel<<<(unsigned)p.tokens, 256, 0, st>>>(c);
}

template <int DT>
void grad_type(const Call& c, hipStream_t st) {
  const Plan& p = c.plan;
  const Head* head = reinterpret_cast<const Head*>(c.ws + p.o_head);
  const u16* h = reinterpret_cast<const u16*>(c.ws + p.o_h);
  u16* gbuf = reinterpret_cast<u16*>(c.ws + p.o_g);
  rows_and_hidden<DT>(c, st);
  for (int64_t v0 = 0; v0 < p.vocab; v0 += p.piece) {
    int64_t ldw;
    const u16* w = piece_weight<DT>(c, v0, &ldw, st);
    const int64_t real = p.vocab - v0 < p.piece ? p.vocab - v0 : p.piece;
    // g of the piece
    Product g = logits_product<DT>(c, w, ldw, real);
    GradEpi<DT> ge{reinterpret_cast<const RowParam*>(c.ws + p.o_rowp), gbuf, p.rows * p.piece,
                   p.piece, 1.0f / c.temperature, (int)v0, (int)real, c.smoothing != 0.0f};
    logits<DT>(p, g, ge, st);
    if (c.k > 0 && p.tokens > 0) entry_kernel<DT><<<(unsigned)p.tokens, 64, 0, st>>>(c, v0);
    // dhidden += g W: the inner index is the piece's vocabulary
    Product d{};
    d.a = {w, p.piece * p.dimp, ldw, (int)p.dimp, (int)real};
    d.b = {gbuf, p.rows * p.piece, p.piece, (int)p.rows, (int)p.piece};
    d.m = (int)p.dimp;
    d.n = (int)p.rows;
    d.inner = round_up_int((int)real, 64);
    d.live_n = true;
    d.segs = g.segs;
    d.split = true;
    d.head = head;
    const SumEpi de{reinterpret_cast<float*>(c.ws + p.o_acc), p.dimp, (int)p.dimp, v0 > 0};
    // dweight of the piece: the inner index is the live rows
    Product e{};
    e.a = {h, p.rows * p.dimp, p.dimp, (int)p.dimp, (int)p.rows};
    e.b = {gbuf, p.rows * p.piece, p.piece, (int)p.piece, (int)p.rows};
    e.m = (int)p.dimp;
    e.n = (int)real;
    e.inner = (int)p.rows;
    e.live_inner = true;
    e.segs = g.segs;
    e.head = head;
    const WeightEpi<DT> we{c.dweight, c.dweight_stride, v0, (int)p.dim,
                           rows_aligned(c.dweight, c.dweight_stride, p.dtype, 8)   ? 8
                           : rows_aligned(c.dweight, c.dweight_stride, p.dtype, 4) ? 4
                                                                                   : 1,
                           head};
    const bool want_d = c.dhidden != nullptr && p.tokens > 0, want_e = c.dweight != nullptr;
    if (p.tokens > kFewTokens) {
      const int64_t across = (p.dimp + 255) / 256;
      const int64_t e_tiles = want_e ? (real + 255) / 256 * across : 0;
      int64_t d_tiles = want_d ? p.rows / 256 * across : 0;
      if (want_d && d_tiles < p.acc_tiles) d_tiles = p.acc_tiles;
      const int first = (int)(e_tiles + 7) / 8 * 8;
      gradients_kernel<DT><<<(unsigned)(first + (d_tiles + 7) / 8 * 8), 512, 0, st>>>(e, we, first,
                                                                                   d, de);
    } else {
      if (want_d) product_tiles<DT, true, false, 256, 64, 2>(d, de, p.acc_tiles, st);
      // at most one inner step, and one stage: what counts is the result's way to
      // memory. fp32's parts are more steps than one
      if (want_e && DT != kF32) product_tiles<DT, true, true, 128, 256, 1>(e, we, 0, st);
      if (want_e && DT == kF32) product_tiles<DT, true, true, 256, 256, 2>(e, we, 0, st);
    }
  }
  if (c.dhidden != nullptr && p.tokens > 0)
    dhidden_kernel<DT><<<dim3((unsigned)p.tokens, (unsigned)((p.dim + 255) / 256)), 64, 0, st>>>(
        c, rows_aligned(c.dhidden, c.dhidden_stride, p.dtype, 4));
}

const char* status() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? nullptr : hipGetErrorString(e);
}

}  // namespace

const char* launch_loss(const Call& c, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (c.plan.dtype == kF32) loss_type<kF32>(c, st);
  else if (c.plan.dtype == kBF16) loss_type<kBF16>(c, st);
  else loss_type<kF16>(c, st);
  return status();
}

const char* launch_grad(const Call& c, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (c.plan.dtype == kF32) grad_type<kF32>(c, st);
  else if (c.plan.dtype == kBF16) grad_type<kBF16>(c, st);
  else grad_type<kF16>(c, st);
  return status();
}

}  // namespace zloss
