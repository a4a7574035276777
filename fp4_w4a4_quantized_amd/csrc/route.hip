// route.hip -- the router of the expert layer (scores, top-k, expert order;
// gradient of the logits) and the combination of the experts' outputs (and
// its gradients).  The operations are defined in include/fp4q.h.
//
// The router is bound by vector instructions and by the chain of its k rounds:
// 16384 x 128, k 8, takes 7.8 us for the choice, 5.6 for the order and 6.2 for the
// gradient (14.0 for the plain softmax's, 370 vector instructions a token of 64-bit
// arithmetic, which issue all the time), where its bytes would take 4 in all; 4096 x
// 256 with groups 11.6 to 12.5 and 5.6 (920 vector instructions a token, 64-bit scores
// among them, which issue in 63% of the cycles).  The combination is bound by HBM:
// 4096 x 8 rows of 2048 (BF16) take 39 us, which also writes back what the call
// before left in the cache, the gradients 48 us (285 MB, 5.9 TB/s); 2047 columns, of
// which a lane takes one at a time, 65 and 94.
#include "fp4q_device.h"
#include "fp4q_internal.h"

namespace fp4q {

namespace {

typedef __bf16 bf16x2r __attribute__((ext_vector_type(2)));
typedef float v2f32r __attribute__((ext_vector_type(2)));

constexpr int RT_TOK = 64;         // most tokens of a workgroup: one bit each in the experts' masks
constexpr int RT_THREADS = 1024;  // 16 waves
constexpr int RT_MAX_E = FP4Q_ROUTE_MAX_EXPERTS;
constexpr int RT_MAX_K = FP4Q_ROUTE_MAX_K;

struct RouteArgs {
  const void* logits;
  int f32;
  int64_t T, ldx;
  int E, k, score, G, top_groups, renorm;
  const float* bias;
  int32_t* experts;
  float* weights;
  int32_t* offsets;
  int32_t* row_src;
  int32_t* row_of;
  uint64_t* masks;  // [blocks][E]: which of the block's tokens chose the expert
  uint8_t* counts;  // [E][pitch]: how many, of each block
  int blocks, tok;  // workgroups and their tokens
  int pitch;        // blocks up to a multiple of 16
  int32_t* before;  // [E][pitch]: rows of the expert in earlier blocks; null: not summed up
  int32_t* total;   // [E]
};

__device__ __forceinline__ float load_value(const void* x, int f32, int64_t i) {
  return f32 ? reinterpret_cast<const float*>(x)[i]
             : bf16_to_f32(reinterpret_cast<const uint16_t*>(x)[i]);
}

// A logit: NaN counts as -inf, +inf as the largest finite number.
__device__ __forceinline__ float logit_of(float x) {
  return x == x ? fminf(x, 0x1.fffffep127f) : -__builtin_inff();
}
__device__ __forceinline__ float load_logit(const void* x, int f32, int64_t i) {
  return logit_of(load_value(x, f32, i));
}

// The logits of experts l, l + STEP, ... of a row that begins at element `row`
// (-inf past the last).  One branch on the type and none on the expert around
// the loads, or each would be waited for before the next is issued.
template <int STEP, int NS>
__device__ __forceinline__ void load_logits(const void* x, int f32, int64_t row, int l, int E,
                                            float (&v)[NS]) {
  if (f32) {
    const float* r = reinterpret_cast<const float*>(x) + row;
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = r[min(l + STEP * i, E - 1)];
  } else {
    const uint16_t* r = reinterpret_cast<const uint16_t*>(x) + row;
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = bf16_to_f32(r[min(l + STEP * i, E - 1)]);
  }
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = l + STEP * i < E ? logit_of(v[i]) : -__builtin_inff();
}

// The value of the lane that differs in bit 0, 1, 2 or 3 of its number (the
// last two: of the mirrored lane, the same for a reduction), by vector moves: a
// shuffle would go through LDS at many times the latency.
template <int BIT>
__device__ __forceinline__ uint32_t lane_swap(uint32_t v) {
  constexpr int ctl = BIT == 0 ? 0xB1 : BIT == 1 ? 0x4E : BIT == 2 ? 0x141 : 0x140;
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctl, 0xF, 0xF, true);
}

template <int BIT>
__device__ __forceinline__ double lane_swap(double v) {
  const u32x2 u = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{lane_swap<BIT>(u[0]), lane_swap<BIT>(u[1])});
}

__device__ __forceinline__ int pick_max(int a, int b) { return a > b ? a : b; }
__device__ __forceinline__ int pick_min(int a, int b) { return a < b ? a : b; }
__device__ __forceinline__ double add(double a, double b) { return a + b; }

// The values of each LANES (16, 32 or 64) lanes joined by f (commutative): every
// lane has the result of its own.
template <typename T, T (*F)(T, T), int LANES>
__device__ __forceinline__ T lanes_all(T v) {
  if constexpr (sizeof(T) == 4) {
    auto bits = [](uint32_t u) { return __builtin_bit_cast(T, u); };
    auto raw = [](T t) { return __builtin_bit_cast(uint32_t, t); };
    v = F(v, bits(lane_swap<0>(raw(v))));
    v = F(v, bits(lane_swap<1>(raw(v))));
    v = F(v, bits(lane_swap<2>(raw(v))));
    v = F(v, bits(lane_swap<3>(raw(v))));
    if constexpr (LANES == 16) return v;
    u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(raw(v), raw(v), false, false));
    v = F(bits(r[0]), bits(r[1]));
    if constexpr (LANES == 32) return v;
    r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(raw(v), raw(v), false, false));
    return F(bits(r[0]), bits(r[1]));
  } else {
    auto bits = [](uint32_t lo, uint32_t hi) { return __builtin_bit_cast(T, u32x2{lo, hi}); };
    u32x2 u = __builtin_bit_cast(u32x2, v);
    v = F(v, bits(lane_swap<0>(u[0]), lane_swap<0>(u[1])));
    u = __builtin_bit_cast(u32x2, v);
    v = F(v, bits(lane_swap<1>(u[0]), lane_swap<1>(u[1])));
    u = __builtin_bit_cast(u32x2, v);
    v = F(v, bits(lane_swap<2>(u[0]), lane_swap<2>(u[1])));
    u = __builtin_bit_cast(u32x2, v);
    v = F(v, bits(lane_swap<3>(u[0]), lane_swap<3>(u[1])));
    if constexpr (LANES == 16) return v;
    u = __builtin_bit_cast(u32x2, v);
    u32x2 l = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(u[0], u[0], false, false));
    u32x2 h = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(u[1], u[1], false, false));
    v = F(bits(l[0], h[0]), bits(l[1], h[1]));
    if constexpr (LANES == 32) return v;
    u = __builtin_bit_cast(u32x2, v);
    l = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(u[0], u[0], false, false));
    h = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(u[1], u[1], false, false));
    return F(bits(l[0], h[0]), bits(l[1], h[1]));
  }
}

template <int LANES = 64, typename T>
__device__ __forceinline__ T wave_max(T v) { return lanes_all<T, pick_max, LANES>(v); }
template <int LANES = 64>
__device__ __forceinline__ int wave_min(int v) { return lanes_all<int, pick_min, LANES>(v); }
template <int LANES = 64>
__device__ __forceinline__ double wave_sum(double v) { return lanes_all<double, add, LANES>(v); }

// Lane l's value, l the same for all lanes.
__device__ __forceinline__ int of_lane(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ double of_lane(double v, int l) {
  const u32x2 u = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{(uint32_t)of_lane((int)u[0], l), (uint32_t)of_lane((int)u[1], l)});
}

// A float as an integer of the same order (both zeros alike; no NaN), and back.
constexpr int ORDER_NONE = (int)0x80000000;  // below every float's
__device__ __forceinline__ int order_of(float x) {
  const int u = __float_as_int(x + 0.0f);
  return u ^ ((u >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float order_value(int o) {
  return __int_as_float(o ^ ((o >> 31) & 0x7FFFFFFF));
}

// The expert order of a workgroup's tokens: base[e] is where the block's
// first row of expert e goes, a token's row among them the number of earlier
// tokens of the block that chose e too.
__device__ __forceinline__ void write_rows(const RouteArgs& p, int64_t t0, int nt,
                                           const int32_t* ex, const uint64_t* mask,
                                           const int* base) {
  for (int i = threadIdx.x; i < nt * p.k; i += blockDim.x) {
    const int t = i / p.k, e = ex[i];
    const int pos = base[e] + (int)__popcll(mask[e] & ((1ull << t) - 1ull));
    p.row_src[pos] = (int32_t)(t0 + t);
    p.row_of[t0 * p.k + i] = pos;
  }
}

// Exclusive scan of n values in LDS by the workgroup (n <= RT_THREADS;
// tmp: one int a wave).
__device__ __forceinline__ void block_scan(int* v, int n, int* tmp, int* total) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int own = t < n ? v[t] : 0;
  int run = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  if (lane == 63) tmp[wave] = run;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < RT_THREADS / 64; ++w) {
    before += w < wave ? tmp[w] : 0;
    all += tmp[w];
  }
  __syncthreads();
  if (t < n) v[t] = before + run - own;
  if (t == 0) *total = all;
  __syncthreads();
}

// One wave per token; lane l holds experts l, l + 64, ...  The order of the
// experts is taken on the logits themselves where they decide it (no bias: both
// scores are increasing functions of the logit), else on the scores in 64 bits,
// so that near ties are told apart as the definition does.  The groups' order
// needs the scores in either case (WIDE: a bias or groups).
template <int NS, bool WIDE>
__global__ __launch_bounds__(RT_THREADS) void k_route_pick(RouteArgs p) {
  __shared__ uint64_t s_mask[RT_MAX_E];
  __shared__ int s_base[RT_MAX_E];
  __shared__ int32_t s_ex[RT_TOK * RT_MAX_K];
  __shared__ int s_tmp[RT_THREADS / 64], s_total;
  extern __shared__ double s_rank[];  // WIDE with groups: [8][E]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = p.E, k = p.k;
  for (int e = threadIdx.x; e < E; e += RT_THREADS) s_mask[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * p.tok;
  const int nt = (int)min((int64_t)p.tok, p.T - t0);
  float next[NS];  // the wave's next token's logits, loaded while one is picked for
  auto load_row = [&](int tt) {
    const int64_t row = (t0 + min(tt, nt - 1)) * p.ldx;
    load_logits<64>(p.logits, p.f32, row, lane, E, next);
  };
  if (wave < nt) load_row(wave);
  for (int tt = wave; tt < nt; tt += RT_THREADS / 64) {
    float x[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) x[i] = next[i];
    load_row(tt + RT_THREADS / 64);
    int ord[NS], top_ord = ORDER_NONE;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      ord[i] = order_of(x[i]);
      top_ord = pick_max(top_ord, ord[i]);
    }
    const float top = order_value(wave_max(top_ord));
    // softmax: scores are exp(x - m) / Z; all scores of a row without a
    // finite logit are 0
    const double m = top > -__builtin_inff() ? (double)top : 0.0;
    const bool soft = p.score == FP4Q_SCORE_SOFTMAX;
    double z = 1.0, s[WIDE ? NS : 1];
    if (WIDE) {
#pragma unroll
      for (int i = 0; i < NS; ++i)
        s[i] = soft ? exp((double)x[i] - m) : 1.0 / (1.0 + exp(-(double)x[i]));
    }
    if (soft && (WIDE || !p.renorm)) {
      double part = 0.0;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (lane + 64 * i < E) part += WIDE ? s[i] : exp((double)x[i] - m);
      z = wave_sum(part);
      if (!(z > 0.0)) z = 1.0;
      if (WIDE) {
#pragma unroll
        for (int i = 0; i < NS; ++i) s[i] /= z;
      }
    }
    // 64-bit keys are compared as integers of the same order, their upper halves
    // first (low: the lower ones); what cannot be picked (any more) has ORDER_NONE
    int key[NS];
    uint32_t low[WIDE ? NS : 1];
    double rank_by[WIDE ? NS : 1];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int e = lane + 64 * i;
      if constexpr (WIDE) {
        double r = s[i] + (p.bias ? (double)p.bias[min(e, E - 1)] : 0.0) + 0.0;
        if (!(r == r)) r = -__builtin_inf();  // NaN comes last
        rank_by[i] = r;
        const u32x2 u = __builtin_bit_cast(u32x2, r);
        const int sign = (int)u[1] >> 31;
        key[i] = p.bias ? (int)u[1] ^ (sign & 0x7FFFFFFF) : ord[i];
        low[i] = p.bias ? u[0] ^ (uint32_t)sign : 0u;
      } else {
        key[i] = ord[i];
      }
      if (e >= E) key[i] = ORDER_NONE;
    }
    if (WIDE && p.G > 1) {
      // each group's two best, by 64 / 2^ceil(log2 G) lanes a group
      double* r = s_rank + wave * E;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (lane + 64 * i < E) r[lane + 64 * i] = rank_by[i];
      wave_fence();
      const int gs = E / p.G;
      int P = 64;
      while (P * p.G > 64) P >>= 1;
      const int g = lane / P;
      double a = -__builtin_inf(), b = -__builtin_inf();
      if (g < p.G)
#pragma unroll 4
        for (int i = lane % P; i < gs; i += P) {
          const double v = r[g * gs + i];
          if (v > a) { b = a; a = v; }
          else if (v > b) b = v;
        }
      auto join = [&](double a2, double b2) {
        const double lo = fmin(a, a2);
        a = fmax(a, a2);
        b = fmax(lo, fmax(b, b2));
      };
      if (P > 1) join(lane_swap<0>(a), lane_swap<0>(b));
      if (P > 2) join(lane_swap<1>(a), lane_swap<1>(b));
      if (P > 4) join(lane_swap<2>(a), lane_swap<2>(b));
      if (P > 8) join(lane_swap<3>(a), lane_swap<3>(b));
      for (int d = 16; d < P; d <<= 1) join(__shfl_xor(a, d), __shfl_xor(b, d));
      double sum = gs > 1 ? a + b : a;
      if (!(sum == sum)) sum = -__builtin_inf();
      int rank = 0;
      for (int o = 0; o < p.G; ++o) {
        const double other = of_lane(sum, o * P);
        rank += (other > sum || (other == sum && o < g)) ? 1 : 0;
      }
      const uint64_t keep = __ballot(g < p.G && rank < p.top_groups);  // a group's P lanes agree
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int e = lane + 64 * i;
        if (e < E && !((keep >> (e / gs * P)) & 1)) key[i] = ORDER_NONE;
      }
      wave_fence();
    }
    // k rounds: the largest key left, the lowest expert that has it; lane j
    // keeps the round's expert and its score
    int my_e = 0;
    for (int j = 0; j < k; ++j) {
      int best = key[0];
#pragma unroll
      for (int i = 1; i < NS; ++i) best = pick_max(best, key[i]);
      best = wave_max(best);
      uint64_t has[NS];
      int n = 0;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        has[i] = __ballot(key[i] == best);
        n += (int)__popcll(has[i]);
      }
      if (WIDE && n > 1) {  // their lower halves decide
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < NS; ++i) most = key[i] == best ? max(most, low[i]) : most;
        // (as signed integers of the same order)
        most = (uint32_t)wave_max((int)(most ^ 0x80000000u)) ^ 0x80000000u;
#pragma unroll
        for (int i = 0; i < NS; ++i) has[i] = __ballot(key[i] == best && low[i] == most);
      }
      int pick = 0;
#pragma unroll
      for (int i = NS - 1; i >= 0; --i)
        if (has[i]) pick = 64 * i + (int)__ffsll((unsigned long long)has[i]) - 1;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (lane + 64 * i == pick) key[i] = ORDER_NONE;
      if (lane == j) my_e = pick;
    }
    double my_s = 0.0;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      double v;
      if constexpr (WIDE) v = __shfl(s[i], my_e & 63);
      else v = (double)__shfl(x[i], my_e & 63);
      if (i == my_e >> 6) my_s = v;
    }
    if (!WIDE) my_s = soft ? exp(my_s - m) / z : 1.0 / (1.0 + exp(-my_s));
    if (p.renorm) {
      const double total = wave_sum(lane < k ? my_s : 0.0);
      my_s = total > 0.0 ? my_s / total : 0.0;
    }
    if (lane < k) {
      p.experts[(t0 + tt) * k + lane] = my_e;
      p.weights[(t0 + tt) * k + lane] = (float)my_s;
      s_ex[tt * k + lane] = my_e;
      atomicOr(reinterpret_cast<uint32_t*>(&s_mask[my_e]) + (tt >> 5), 1u << (tt & 31));
    }
  }
  __syncthreads();
  if (p.blocks > 1) {
    for (int e = threadIdx.x; e < E; e += RT_THREADS) {
      p.masks[(int64_t)blockIdx.x * E + e] = s_mask[e];
      p.counts[(int64_t)e * p.pitch + blockIdx.x] = (uint8_t)__popcll(s_mask[e]);
    }
    return;
  }
  for (int e = threadIdx.x; e < E; e += RT_THREADS) s_base[e] = (int)__popcll(s_mask[e]);
  __syncthreads();
  block_scan(s_base, E, s_tmp, &s_total);
  for (int e = threadIdx.x; e < E; e += RT_THREADS) p.offsets[e] = s_base[e];
  if (threadIdx.x == 0) p.offsets[E] = s_total;
  write_rows(p, t0, nt, s_ex, s_mask, s_base);
}

// The same without bias and groups for k up to 16 and more tokens than one
// workgroup has: 16 lanes per token, lane l with experts l, l + 16, ..., so that
// four tokens share each exchange between lanes and each 64-bit exponential
// (x 128 experts, k 8, the order included: 4096 tokens 9.3 us, by one wave a token
// 10.2).
template <int NS>
__global__ __launch_bounds__(RT_THREADS) void k_route_pick16(RouteArgs p) {
  __shared__ uint64_t s_mask[RT_MAX_E];
  const int E = p.E, k = p.k, l = threadIdx.x & 15, tt = threadIdx.x >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * p.tok;
  const int nt = (int)min((int64_t)p.tok, p.T - t0);
  float x[NS];
  load_logits<16>(p.logits, p.f32, (t0 + min(tt, nt - 1)) * p.ldx, l, E, x);
  for (int e = threadIdx.x; e < E; e += blockDim.x) s_mask[e] = 0;
  __syncthreads();
  int key[NS], best = ORDER_NONE;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    key[i] = l + 16 * i < E ? order_of(x[i]) : ORDER_NONE;
    best = pick_max(best, key[i]);
  }
  const float top = order_value(wave_max<16>(best));
  const double m = top > -__builtin_inff() ? (double)top : 0.0;
  const bool soft = p.score == FP4Q_SCORE_SOFTMAX;
  double z = 1.0;
  if (soft && !p.renorm) {
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (l + 16 * i < E) part += exp((double)order_value(key[i]) - m);
    z = wave_sum<16>(part);
    if (!(z > 0.0)) z = 1.0;
  }
  int my_e = 0, my_key = 0;
  for (int j = 0; j < k; ++j) {
    best = key[0];
#pragma unroll
    for (int i = 1; i < NS; ++i) best = pick_max(best, key[i]);
    best = wave_max<16>(best);
    int at = NS;
#pragma unroll
    for (int i = NS - 1; i >= 0; --i) at = key[i] == best ? i : at;
    const int pick = wave_min<16>(16 * at + l);
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (pick == 16 * i + l) key[i] = ORDER_NONE;
    if (l == j) {
      my_e = pick;
      my_key = best;
    }
  }
  const double my_x = (double)order_value(my_key);
  double my_s = soft ? exp(my_x - m) / z : 1.0 / (1.0 + exp(-my_x));
  if (p.renorm) {
    const double total = wave_sum<16>(l < k ? my_s : 0.0);
    my_s = total > 0.0 ? my_s / total : 0.0;
  }
  if (l < k && tt < nt) {
    p.experts[(t0 + tt) * k + l] = my_e;
    p.weights[(t0 + tt) * k + l] = (float)my_s;
    atomicOr(reinterpret_cast<uint32_t*>(&s_mask[my_e]) + (tt >> 5), 1u << (tt & 31));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    p.masks[(int64_t)blockIdx.x * E + e] = s_mask[e];
    p.counts[(int64_t)e * p.pitch + blockIdx.x] = (uint8_t)__popcll(s_mask[e]);
  }
}

// Sums up the counts of the blocks before each one, a workgroup an expert: a
// lane takes 16 blocks at a time.
__global__ __launch_bounds__(RT_THREADS) void k_route_sums(RouteArgs p) {
  __shared__ int s_sum[RT_THREADS], s_tmp[RT_THREADS / 64], s_total;
  const int64_t row = (int64_t)blockIdx.x * p.pitch;
  int before = 0;
  for (int c0 = 0; c0 < p.blocks; c0 += RT_THREADS * 16) {
    const int c = c0 + threadIdx.x * 16;
    u32x4 w = {0, 0, 0, 0};
    if (c < p.blocks) w = *reinterpret_cast<const u32x4*>(p.counts + row + c);
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = p.blocks - c - 4 * i;
      w[i] &= n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
      own = __builtin_amdgcn_sad_u8(w[i], 0u, own);
    }
    s_sum[threadIdx.x] = (int)own;
    __syncthreads();
    block_scan(s_sum, RT_THREADS, s_tmp, &s_total);
    int run = before + s_sum[threadIdx.x];
    if (c < p.blocks) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p.before[row + c + i] = run;  // (the row's padding included)
        run += (w[i >> 2] >> (8 * (i & 3))) & 0xFF;
      }
    }
    before += s_total;
    __syncthreads();
  }
  if (threadIdx.x == 0) p.total[blockIdx.x] = before;
}

// Expert order over all workgroups' tokens: a workgroup sums every block's
// counts (all of them for the experts' offsets, the earlier blocks' for its
// own base) and places its rows.  Q neighbouring lanes share an expert's counts,
// 16 bytes at a time.  With many blocks, where that would grow with their
// square, k_route_sums has done it.
__global__ __launch_bounds__(RT_THREADS) void k_route_order(RouteArgs p) {
  __shared__ int s_base[RT_MAX_E], s_before[RT_MAX_E];
  __shared__ int s_tmp[RT_THREADS / 64], s_total;
  __shared__ uint64_t s_mask[RT_MAX_E];
  const int E = p.E;
  const int64_t t0 = (int64_t)blockIdx.x * p.tok;
  const int nt = (int)min((int64_t)p.tok, p.T - t0);
  int Q = 64;
  while (Q * E > RT_THREADS && Q > 1) Q >>= 1;
  const int q = threadIdx.x % Q;
  if (p.before) {
    for (int e = threadIdx.x; e < E; e += RT_THREADS) {
      s_base[e] = p.total[e];
      s_before[e] = p.before[(int64_t)e * p.pitch + blockIdx.x];
      s_mask[e] = p.masks[(int64_t)blockIdx.x * E + e];
    }
  } else for (int e = threadIdx.x / Q; e < E; e += RT_THREADS / Q) {
    uint32_t all = 0, before = 0;
    for (int c = q * 16; c < p.blocks; c += Q * 16) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(p.counts + (int64_t)e * p.pitch + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the bytes of the first n of these four blocks
        auto first = [&](int n) { return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u; };
        all = __builtin_amdgcn_sad_u8(w[i] & first(p.blocks - c - 4 * i), 0u, all);
        before = __builtin_amdgcn_sad_u8(w[i] & first((int)blockIdx.x - c - 4 * i), 0u, before);
      }
    }
    for (int d = 1; d < Q; d <<= 1) {
      all += __shfl_xor(all, d);
      before += __shfl_xor(before, d);
    }
    if (q == 0) {
      s_base[e] = (int)all;
      s_before[e] = (int)before;
      s_mask[e] = p.masks[(int64_t)blockIdx.x * E + e];
    }
  }
  __syncthreads();
  block_scan(s_base, E, s_tmp, &s_total);
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < E; e += RT_THREADS) p.offsets[e] = s_base[e];
    if (threadIdx.x == 0) p.offsets[E] = s_total;
  }
  for (int e = threadIdx.x; e < E; e += RT_THREADS) s_base[e] += s_before[e];
  __syncthreads();
  write_rows(p, t0, nt, p.experts + t0 * p.k, s_mask, s_base);
}

struct GradArgs {
  const void* logits;
  int f32;
  int64_t T, ldx;
  int E, k, score, renorm;
  const int32_t* experts;
  const float* dw;
  void* d;
  int64_t ldd;
};

// The gradients of experts l, l + STEP, ... of token t.
template <int STEP, int NS>
__device__ __forceinline__ void store_gradient(const GradArgs& p, int64_t t, int l, const float (&v)[NS]) {
  if (p.f32) {
    float* r = reinterpret_cast<float*>(p.d) + t * p.ldd;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (l + STEP * i < p.E) r[l + STEP * i] = v[i];
  } else {
    __bf16* r = reinterpret_cast<__bf16*>(p.d) + t * p.ldd;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (l + STEP * i < p.E) r[l + STEP * i] = (__bf16)v[i];
  }
}

// Gradient of the logits.  With p the chosen scores and dp their gradient:
//   softmax: dx_i = -score_i sum(dp p), plus dp_i score_i where chosen
//   sigmoid: dx_i = dp_i score_i (1 - score_i) where chosen, else 0
// Through the renormalisation w = p / sum p it is dp = (dw - sum(dw w)) / sum p,
// for which sum(dp p) = 0: then the softmax's sum over all experts cancels and
// the chosen logits' exponentials (relative to the largest logit, as the scores
// have them) are all that is needed.  So it is with all but the plain softmax:
// LANES lanes per token, lane j with the j-th chosen expert, whose gradients
// meet the zeros of the others in LDS (an expert that is named twice in the
// order of j).  16384 x 128, k 8 take 6.3 us (17 MB, of which 3 us), with one
// wave per token and one load after another 13.3.
template <int LANES, int NS>
__global__ __launch_bounds__(256) void k_route_backward(GradArgs p) {
  extern __shared__ float s_dx[];  // [256 / LANES][E]
  const int l = threadIdx.x % LANES, E = p.E, k = p.k;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t t = block * (256 / LANES) + threadIdx.x / LANES;
  if (t >= p.T) return;
  float* const dx = s_dx + threadIdx.x / LANES * E;
  const bool soft = p.score == FP4Q_SCORE_SOFTMAX;
  const int e = l < k ? p.experts[t * k + l] : -1;
  const bool on = e >= 0 && e < E;  // (an index outside the experts: no gradient)
  const float given = l < k ? p.dw[t * k + l] : 0.0f;
  float row[NS];
  if (soft) load_logits<LANES>(p.logits, p.f32, t * p.ldx, l, E, row);
  for (int c = l; c < E; c += LANES) dx[c] = 0.0f;
  const double x = on ? (double)load_logit(p.logits, p.f32, t * p.ldx + e) : 0.0;
  double dw = on ? (double)given : 0.0, m = 0.0;
  if (soft) {
    int top = ORDER_NONE;
#pragma unroll
    for (int i = 0; i < NS; ++i) top = pick_max(top, order_of(row[i]));
    const float v = order_value(wave_max<LANES>(top));
    if (v > -__builtin_inff()) m = (double)v;
  }
  double s = 0.0;
  if (on) s = soft ? exp(x - m) : 1.0 / (1.0 + exp(-x));
  if (p.renorm) {
    const double sum = wave_sum<LANES>(s), dot = wave_sum<LANES>(dw * s);
    const double r = sum > 0.0 ? 1.0 / sum : 0.0;
    dw = (dw - dot * r) * r;
  }
  const float mine = (float)(soft ? dw * s : dw * s * (1.0 - s));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  // (a wave's LDS operations keep their order)
  for (int j = 0; j < k; ++j)
    if (l == j && on) __hip_atomic_fetch_add(&dx[e], mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  float out[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) out[i] = dx[min(l + LANES * i, E - 1)];
  store_gradient<LANES>(p, t, l, out);
}

// The plain softmax's, one wave per token: it needs all scores.
template <int NS>
__global__ __launch_bounds__(256) void k_route_backward_softmax(GradArgs p) {
  const int lane = threadIdx.x & 63, E = p.E, k = p.k;
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  float x[NS];
  load_logits<64>(p.logits, p.f32, t * p.ldx, lane, E, x);
  int top_ord = ORDER_NONE;
#pragma unroll
  for (int i = 0; i < NS; ++i) top_ord = pick_max(top_ord, order_of(x[i]));
  const float top = order_value(wave_max(top_ord));
  const double m = top > -__builtin_inff() ? (double)top : 0.0;
  // lane j: the j-th chosen expert (indices outside the experts: no gradient)
  const int e = lane < k ? p.experts[t * k + lane] : -1;
  const bool on = e >= 0 && e < E;
  const double dw = on ? (double)p.dw[t * k + lane] : 0.0;
  double s[NS], part = 0.0;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    s[i] = lane + 64 * i < E ? exp((double)x[i] - m) : 0.0;
    part += s[i];
  }
  double z = wave_sum(part);
  z = z > 0.0 ? 1.0 / z : 1.0;
  double mine = 0.0;  // dw p of lane j's expert
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    s[i] *= z;
    const double si = __shfl(s[i], e & 63);
    if (on && i == e >> 6) mine = dw * si;
  }
  const double dot = wave_sum(mine);
  double dx[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) dx[i] = -s[i] * dot;
  for (int j = 0; j < k; ++j) {
    const int ej = of_lane(e, j);
    const double aj = of_lane(mine, j);
    const double add_e = (ej & 63) == lane ? aj : 0.0;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (i == ej >> 6) dx[i] += add_e;  // (of ej < 0: none)
  }
  float out[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) out[i] = (float)dx[i];
  store_gradient<64>(p, t, lane, out);
}

// ---- the combination --------------------------------------------------------

// VEC consecutive values as f32: 8 BF16 (16 bytes) or 4 F32, or one of either.
template <bool F32, int VEC>
__device__ __forceinline__ void load_vec(const void* x, int64_t i, float (&v)[VEC]) {
  if (VEC == 1) {
    v[0] = load_value(x, F32, i);
  } else if (F32) {
#pragma unroll
    for (int c = 0; c < VEC / 4; ++c) {
      const u32x4 u = reinterpret_cast<const u32x4*>(reinterpret_cast<const float*>(x) + i)[c];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * c + e] = __uint_as_float(u[e]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < VEC / 8; ++c) {
      const u32x4 u = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(x) + i)[c];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[8 * c + 2 * e] = __uint_as_float(u[e] << 16);
        v[8 * c + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      }
    }
  }
}

template <bool F32, int VEC>
__device__ __forceinline__ void store_vec(void* y, int64_t i, const float (&v)[VEC]) {
  if (VEC == 1) {
    if (F32) reinterpret_cast<float*>(y)[i] = v[0];
    else reinterpret_cast<__bf16*>(y)[i] = (__bf16)v[0];
  } else if (F32) {
#pragma unroll
    for (int c = 0; c < VEC / 4; ++c) {
      u32x4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = __float_as_uint(v[4 * c + e]);
      reinterpret_cast<u32x4*>(reinterpret_cast<float*>(y) + i)[c] = u;
    }
  } else {
#pragma unroll
    for (int c = 0; c < VEC / 8; ++c) {
      u32x4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const v2f32r f = {v[8 * c + 2 * e], v[8 * c + 2 * e + 1]};
        u[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2r));
      }
      reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(y) + i)[c] = u;
    }
  }
}

struct CombineArgs {
  const void* y;
  int64_t rows, N, ldy;
  const int32_t* row_of;
  const float* w;
  int64_t T;
  int k;
  void* out;
  int64_t ldo;
  const void* d_out;
  void* d_y;
  int64_t lddy;
  float* d_w;
  int32_t* named;  // [rows], null: not asked for; the entry of row_of that names the row
};

// out[t] = sum_j w[t, j] y[row_of[t, j]]: a thread holds VEC columns of one
// token, the rows added in order j in FP32, eight rows' loads in flight (an
// entry outside the rows loads row 0 and adds nothing).
template <bool F32, int VEC>
__global__ __launch_bounds__(256) void k_combine(CombineArgs p) {
  const int64_t per = p.N / VEC;
  const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.T * per) return;
  const int64_t t = i / per, c = (i - t * per) * VEC;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
  for (int j0 = 0; p.rows > 0 && j0 < p.k; j0 += 8) {
    float v[8][VEC], w[8];
    bool ok[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = min(j0 + u, p.k - 1);
      const int32_t r = p.row_of[t * p.k + j];
      ok[u] = j0 + u < p.k && r >= 0 && r < p.rows;
      w[u] = p.w[t * p.k + j];
      load_vec<F32, VEC>(p.y, (ok[u] ? r : 0) * p.ldy + c, v[u]);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = ok[u] ? __builtin_fmaf(w[u], v[u][e], acc[e]) : acc[e];
  }
  store_vec<F32, VEC>(p.out, t * p.ldo + c, acc);
}

// d_y[row_of[t, j]] = w[t, j] d_out[t], d_w[t, j] = y[row_of[t, j]] . d_out[t]:
// one wave per (token, j), the products summed in FP32.
template <bool F32, int VEC>
__global__ __launch_bounds__(256) void k_combine_backward(CombineArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (i >= p.T * p.k) return;
  const int64_t t = i / p.k, r = p.row_of[i];
  if (r < 0 || r >= p.rows) {
    if (lane == 0) p.d_w[i] = 0.0f;
    return;
  }
  if (p.named && lane == 0) p.named[r] = (int32_t)i;
  const float w = p.w[i];
  float dot = 0.0f;
  for (int64_t c = (int64_t)lane * VEC; c < p.N; c += 64 * VEC) {
    float v[VEC], d[VEC];
    load_vec<F32, VEC>(p.y, r * p.ldy + c, v);
    load_vec<F32, VEC>(p.d_out, t * p.ldo + c, d);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      dot = __builtin_fmaf(v[e], d[e], dot);
      d[e] *= w;
    }
    store_vec<F32, VEC>(p.d_y, r * p.lddy + c, d);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
  if (lane == 0) p.d_w[i] = dot;
}

// The rows of d_y that no entry of row_of names become 0, a wave for 64 rows.
// named[] was not cleared before k_combine_backward wrote it: what it holds for
// a row counts where row_of bears it out, and then the row is named, whoever
// wrote it.  (Zeroing all of d_y first would write it twice: 134 MB for 4096 x 8 rows
// of 2048 in BF16, at least 27 us, where this launch adds 2.8 to the pass.)
template <bool F32, int VEC>
__global__ __launch_bounds__(256) void k_zero_unnamed(CombineArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t r0 = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6)) * 64;
  const int64_t r = r0 + lane;
  bool rest = false;
  if (r < p.rows) {
    const int64_t i = p.named[r];
    rest = i < 0 || i >= p.T * p.k || p.row_of[i] != r;
  }
  float zero[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) zero[e] = 0.0f;
  for (uint64_t left = __ballot(rest); left; left &= left - 1) {
    const int64_t at = (r0 + __ffsll((unsigned long long)left) - 1) * p.lddy;
    for (int64_t c = (int64_t)lane * VEC; c < p.N; c += 64 * VEC) store_vec<F32, VEC>(p.d_y, at + c, zero);
  }
}

// A grid of n workgroups of 256, in rows: one dimension holds 2^32 threads.
inline dim3 grid_of(int64_t n) {
  const int64_t x = n < 1 ? 1 : n < (1 << 20) ? n : 1 << 20;
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

inline bool vec_ok(const void* p, int64_t ld, int esz) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * esz) % 16 == 0;
}

}  // namespace

// Tokens of a workgroup: few while that leaves CUs without one (x 256 experts, k 8:
// 4096 tokens 11.7 us a call by 16 and 13.6 by 64, in 8 groups 16.7 and 34.8;
// 16384 tokens 21.4 and 16.5, in groups 49.4 and 38.0).
static int route_tokens(int64_t T) { return T <= 256 * 16 ? 16 : T <= 256 * 32 ? 32 : RT_TOK; }

// Blocks from which on their counts are summed up by a kernel of its own
// (x 128 experts, k 8: 256 blocks 12.3 us a call without it and 14.1 with it, 512
// 20.4 and 18.7, 1024 43.9 and 31.0).
constexpr int RT_SUMS = 512;

size_t route_workspace_bytes(int64_t T, int E) {
  const int64_t tok = route_tokens(T), blocks = (T + tok - 1) / tok, pitch = (blocks + 15) / 16 * 16;
  if (blocks <= 1) return 0;
  return (size_t)E * (size_t)(pitch + blocks * 8 + (blocks >= RT_SUMS ? (pitch + 1) * 4 : 0));
}

void launch_route(const void* logits, int f32, int64_t T, int64_t ldx, int E, int k, int score,
                  const float* bias, int G, int top_groups, int renorm, int32_t* experts,
                  float* weights, int32_t* offsets, int32_t* row_src, int32_t* row_of, void* ws,
                  hipStream_t stream) {
  const int tok = route_tokens(T), blocks = (int)((T + tok - 1) / tok);
  RouteArgs p = {logits,  f32,     T,       ldx,     E,      k,  score, G, top_groups, renorm, bias,
                 experts, weights, offsets, row_src, row_of, nullptr, nullptr, blocks > 0 ? blocks : 1,
                 tok,     (blocks + 15) / 16 * 16, nullptr, nullptr};
  if (blocks > 1) {
    p.counts = static_cast<uint8_t*>(ws);
    p.masks = reinterpret_cast<uint64_t*>(p.counts + (int64_t)E * p.pitch);
    if (blocks >= RT_SUMS) {
      p.before = reinterpret_cast<int32_t*>(p.masks + (int64_t)blocks * E);
      p.total = p.before + (int64_t)E * p.pitch;
    }
  }
  const bool wide = bias != nullptr || G > 1;
  const dim3 grid((unsigned)p.blocks), thr(RT_THREADS);
  const size_t lds = G > 1 ? (size_t)(RT_THREADS / 64) * E * sizeof(double) : 0;
#define FP4Q_ROUTE(N)                                                                    \
  if (wide) hipLaunchKernelGGL((k_route_pick<N, true>), grid, thr, lds, stream, p);      \
  else hipLaunchKernelGGL((k_route_pick<N, false>), grid, thr, 0, stream, p)
#define FP4Q_ROUTE16(N) hipLaunchKernelGGL((k_route_pick16<N>), grid, dim3(16 * tok), 0, stream, p)
  if (!wide && blocks > 1 && k <= 16) {
    if (E <= 64) FP4Q_ROUTE16(4);
    else if (E <= 128) FP4Q_ROUTE16(8);
    else if (E <= 256) FP4Q_ROUTE16(16);
    else FP4Q_ROUTE16(32);
  }
  else if (E <= 64) { FP4Q_ROUTE(1); }
  else if (E <= 128) { FP4Q_ROUTE(2); }
  else if (E <= 256) { FP4Q_ROUTE(4); }
  else { FP4Q_ROUTE(8); }
#undef FP4Q_ROUTE
#undef FP4Q_ROUTE16
  if (p.before) hipLaunchKernelGGL(k_route_sums, dim3((unsigned)E), thr, 0, stream, p);
  if (blocks > 1) hipLaunchKernelGGL(k_route_order, grid, thr, 0, stream, p);
}

void launch_route_backward(const void* logits, int f32, int64_t T, int64_t ldx, int E, int k,
                           int score, int renorm, const int32_t* experts, const float* d_weights,
                           void* d_logits, int64_t ldd, hipStream_t stream) {
  const GradArgs p = {logits, f32, T, ldx, E, k, score, renorm, experts, d_weights, d_logits, ldd};
  const int lanes = score == FP4Q_SCORE_SOFTMAX && !renorm ? 64 : k <= 16 ? 16 : 32;
  const int per = 256 / lanes;
  const dim3 grid = grid_of((T + per - 1) / per), thr(256);
  const size_t lds = (size_t)per * E * sizeof(float);
#define FP4Q_SOFTMAX(N) hipLaunchKernelGGL((k_route_backward_softmax<N>), grid, thr, 0, stream, p)
#define FP4Q_GRAD(L, N) hipLaunchKernelGGL((k_route_backward<L, N>), grid, thr, lds, stream, p)
  if (lanes == 64) {
    if (E <= 64) FP4Q_SOFTMAX(1);
    else if (E <= 128) FP4Q_SOFTMAX(2);
    else if (E <= 256) FP4Q_SOFTMAX(4);
    else FP4Q_SOFTMAX(8);
  } else if (lanes == 32) {
    FP4Q_GRAD(32, RT_MAX_E / 32);
  } else {
    if (E <= 64) FP4Q_GRAD(16, 4);
    else if (E <= 128) FP4Q_GRAD(16, 8);
    else if (E <= 256) FP4Q_GRAD(16, 16);
    else FP4Q_GRAD(16, 32);
  }
#undef FP4Q_SOFTMAX
#undef FP4Q_GRAD
}

void launch_combine(int f32, const void* y, int64_t rows, int64_t N, int64_t ldy,
                    const int32_t* row_of, const float* w, int64_t T, int k, void* out,
                    int64_t ldo, hipStream_t stream) {
  const CombineArgs p = {y, rows, N, ldy, row_of, w, T, k, out, ldo, nullptr, nullptr, 0, nullptr, nullptr};
  const int esz = f32 ? 4 : 2;
  const bool vec = N % 8 == 0 && vec_ok(y, ldy, esz) && vec_ok(out, ldo, esz);
  const int64_t items = T * (vec ? N / 8 : N);
  const dim3 grid = grid_of((items + 255) / 256), thr(256);
  if (f32) {
    if (vec) hipLaunchKernelGGL((k_combine<true, 8>), grid, thr, 0, stream, p);
    else hipLaunchKernelGGL((k_combine<true, 1>), grid, thr, 0, stream, p);
  } else {
    if (vec) hipLaunchKernelGGL((k_combine<false, 8>), grid, thr, 0, stream, p);
    else hipLaunchKernelGGL((k_combine<false, 1>), grid, thr, 0, stream, p);
  }
}

void launch_combine_backward(int f32, const void* y, int64_t rows, int64_t N, int64_t ldy,
                             const int32_t* row_of, const float* w, int64_t T, int k,
                             const void* d_out, int64_t ldo, void* d_y, int64_t lddy, float* d_w,
                             int32_t* named, hipStream_t stream) {
  const CombineArgs p = {y,       rows, N,     ldy, row_of, w,    T,
                         k,       nullptr, ldo, d_out, d_y, lddy, d_w, named};
  const int esz = f32 ? 4 : 2;
  const bool vec = N % 8 == 0 && vec_ok(y, ldy, esz) && vec_ok(d_out, ldo, esz) &&
                   vec_ok(d_y, lddy, esz);
  const dim3 thr(256), grid = grid_of((T * k + 3) / 4), rest = grid_of((rows + 255) / 256);
#define FP4Q_GRADIENT(F, V)                                                                        \
  do {                                                                                             \
    if (T > 0) hipLaunchKernelGGL((k_combine_backward<F, V>), grid, thr, 0, stream, p);            \
    if (named && rows > 0) hipLaunchKernelGGL((k_zero_unnamed<F, V>), rest, thr, 0, stream, p);    \
  } while (0)
  if (f32) {
    if (vec) FP4Q_GRADIENT(true, 8);
    else FP4Q_GRADIENT(true, 1);
  } else {
    if (vec) FP4Q_GRADIENT(false, 8);
    else FP4Q_GRADIENT(false, 1);
  }
#undef FP4Q_GRADIENT
}

}  // namespace fp4q
