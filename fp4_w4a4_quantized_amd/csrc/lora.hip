// lora.hip -- low-rank adapters of many requests beside a shared projection
// (defined in include/fp4q.h): for the rows of each request,
//   out = y + s (x A^T) B^T   with its adapter's A [rank, K], B [N, rank].
//
// Bound by HBM: y is read and written once, x read once (prompts), or the
// adapters' A and B, which a request of one token reads whole (decode).  8192 rows
// of 11 requests, rank 32, K 4096, N 14336 (BF16, 536 MB): 22 + 114 us, 3.9 TB/s of the
// 4.7 of a copy; 64 requests of one row with 37 adapters of rank 16 (26 MB): 4.3 + 9.6,
// the chain of a search, three loads and the sums in each.  Two
// kernels: u = x A^T with K split over the waves and, where there are few rows,
// over workgroups (partial sums in F32, added in order by the second kernel);
// then out, each workgroup some columns of a tile of rows.
//
// Products are 16x16x32 on BF16.  x, A and B enter as they are; u enters the
// second product as two BF16 terms (u but for 2^-17) where out is BF16, as three
// (2^-25) where it is F32: one term, 2^-9, would be as large as out's own rounding.
// An infinite element of B meets each term by itself, so a step's sums are looked at
// and, where one is infinite or NaN, taken again: 64 requests of one row 13.4 to 13.7 us,
// the 8192 rows 141.8 to 143.0 (both calls back to back, three inputs in turn).
#include "fp4q_device.h"
#include "fp4q_internal.h"

namespace fp4q {

namespace {

typedef float f32x4l __attribute__((ext_vector_type(4)));
typedef float f32x2l __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2l __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8l __attribute__((ext_vector_type(8)));
// Sixteen bytes at any element's address (rows of odd strides).
typedef uint32_t u32x4_2l __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_4l __attribute__((ext_vector_type(4), aligned(4)));

constexpr float BF16_MAX = 0x1.FEp127f;  // the largest finite one
constexpr int U_MT = 4, U_MT_128 = 2, OUT_MT = 2;  // products of a tile of many rows (U_MT_128: ranks above 64)

struct LoraArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;  // or null: 1
  int adapters, rank;
  const int32_t* off;
  const int32_t* adapter;
  int G;
  int64_t rows;
  int64_t K, N;
  const void* y;       // or null: 0
  int64_t ldy;
  void* out;
  int64_t ldo;
  float* u;            // [splits][rows][ur]
  int ur;
  int splits;
  int64_t chunk;       // of K, a split's
  int iters, parts;    // 256-column steps of a workgroup, workgroups of a tile
};

// The rows of a workgroup: `n` from row r0, of adapter `a` (-1: none).
struct LoraTile {
  int64_t r0;
  int n, a;
};

// Sum of v over the lanes up to this one, by vector moves: within 16 lanes, then
// the last of each 16 added to the next, and of the lower 32 to the upper.
__device__ __forceinline__ int sum_to_lane(int v) {
#define FP4Q_SHIFT(CTRL, ROWS) v += __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
  FP4Q_SHIFT(0x111, 0xF)  // one lane up
  FP4Q_SHIFT(0x112, 0xF)
  FP4Q_SHIFT(0x114, 0xF)
  FP4Q_SHIFT(0x118, 0xF)
  FP4Q_SHIFT(0x142, 0xA)  // lane 15 of a row to the next row
  FP4Q_SHIFT(0x143, 0xC)  // lane 31 to the upper half
#undef FP4Q_SHIFT
  return v;
}

// Tile number `tile` when each request's rows are cut into tiles of TM; after
// the last request come the rows of none.  By a whole wave, 64 requests a step.
template <int TM>
__device__ __forceinline__ LoraTile lora_tile(const LoraArgs& p, int tile) {
  const int lane = threadIdx.x & 63, rows = (int)p.rows;
  LoraTile t = {0, 0, -1};
  int before = 0;
  for (int g0 = 0; g0 <= p.G; g0 += 64) {
    const int g = g0 + lane;
    // (loads side by side, of some request where there is none)
    const int o0 = p.off[min(g, p.G)], o1 = p.off[min(g + 1, p.G)], o2 = p.adapter[min(g, p.G - 1)];
    const int r0 = g <= p.G ? min(max(o0, 0), rows) : rows;
    const int r1 = g < p.G ? min(max(o1, r0), rows) : rows;
    const int id = g < p.G ? o2 : -1;
    const int mine = (r1 - r0 + TM - 1) / TM;
    const int to = before + sum_to_lane(mine), first = to - mine;  // of this request's tiles
    const uint64_t hit = __ballot(tile >= first && tile < to);
    if (hit) {
      const int at = __ffsll((unsigned long long)hit) - 1;
      auto of = [&](int v) { return __builtin_amdgcn_readlane(v, at); };
      const int64_t from = of(r0) + (int64_t)(tile - of(first)) * TM;
      if (from < of(r0) || from >= of(r1)) return t;  // (offsets that go down could lead here)
      t.r0 = from;
      t.n = min(TM, of(r1) - (int)from);
      t.a = of(id);
      if (t.a < 0 || t.a >= p.adapters) t.a = -1;
      return t;
    }
    before = __builtin_amdgcn_readlane(to, 63);
  }
  return t;
}

__device__ __forceinline__ f32x4l product(u32x4 a, u32x4 b, f32x4l c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8l, a), __builtin_bit_cast(bf16x8l, b),
                                                 c, 0, 0, 0);
}

// u of a tile of 16 MT rows: A's rows (ranks) by x's rows.  A lane has, of one
// row, ranks 4 (lane / 16) .. + 3 of each 16.
template <int MT, int RT>
__global__ __launch_bounds__(256) void k_lora_u(LoraArgs p) {
  constexpr int TM = 16 * MT;
  __shared__ f32x4l s_acc[4][MT * RT][64];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const LoraTile t = lora_tile<TM>(p, blockIdx.x);
  if (t.n == 0 || t.a < 0) return;
  const int64_t k0 = blockIdx.y * p.chunk, k1 = min(p.K, k0 + p.chunk);
  // (of ranks and rows that are not there the last one's: what comes of them is not used)
  const uint16_t* a[RT];
  const uint16_t* x[MT];
#pragma unroll
  for (int i = 0; i < RT; ++i) a[i] = p.a + ((int64_t)t.a * p.rank + min(16 * i + c, p.rank - 1)) * p.K;
#pragma unroll
  for (int i = 0; i < MT; ++i) x[i] = p.x + (t.r0 + min(16 * i + c, t.n - 1)) * p.ldx;
  f32x4l acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[m][i] = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = MT * RT >= 32 ? 1 : MT * RT >= 8 ? 2 : 4;  // steps of 32 along K that are loaded together
  struct Batch {
    u32x4 a[U][RT], x[U][MT];
  };
  // Loads without conditions, so that none waits for another: past the split's
  // end its first ones again, which count as 0 on both sides (an infinity among them).
  auto load = [&](Batch& f, int64_t k) {
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int64_t at = k + 32 * s + 8 * g < k1 ? k + 32 * s + 8 * g : k0;  // (K and a split's end: multiples of 8)
#pragma unroll
      for (int i = 0; i < RT; ++i) f.a[s][i] = *reinterpret_cast<const u32x4*>(a[i] + at);
#pragma unroll
      for (int m = 0; m < MT; ++m) f.x[s][m] = *reinterpret_cast<const u32x4*>(x[m] + at);
    }
  };
  auto multiply = [&](Batch& f, int64_t k) {
    if (k + 32 * U > k1) {
#pragma unroll
      for (int s = 0; s < U; ++s)
        if (k + 32 * s + 8 * g >= k1) {
#pragma unroll
          for (int i = 0; i < RT; ++i) f.a[s][i] = u32x4{0, 0, 0, 0};
#pragma unroll
          for (int m = 0; m < MT; ++m) f.x[s][m] = u32x4{0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[m][i] = product(f.a[s][i], f.x[s][m], acc[m][i]);
  };
  // the next batch on its way while one is multiplied
  constexpr int64_t STRIDE = 128 * U;
  Batch f0, f1;
  int64_t k = k0 + wave * (32 * U);
  if (k < k1) load(f0, k);
  for (; k < k1; k += 2 * STRIDE) {
    if (k + STRIDE < k1) load(f1, k + STRIDE);
    multiply(f0, k);
    if (k + STRIDE >= k1) break;
    if (k + 2 * STRIDE < k1) load(f0, k + 2 * STRIDE);
    multiply(f1, k + STRIDE);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < RT; ++i) s_acc[wave][m * RT + i][lane] = acc[m][i];
  __syncthreads();
  float* u = p.u + (int64_t)blockIdx.y * p.rows * p.ur;
  for (int j = wave; j < MT * RT; j += 4) {
    f32x4l v = s_acc[0][j][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += s_acc[w][j][lane];
    const int row = 16 * (j / RT) + c;
    if (row < t.n) *reinterpret_cast<f32x4l*>(u + (t.r0 + row) * p.ur + 16 * (j % RT) + 4 * g) = v;
  }
}

// Eight BF16 with 0 for those that are infinite or NaN.
__device__ __forceinline__ u32x4 finite_of(u32x4 v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & 0x7F80u) == 0x7F80u) v[i] &= 0xFFFF0000u;
    if ((v[i] & 0x7F800000u) == 0x7F800000u) v[i] &= 0xFFFFu;
  }
  return v;
}

// Sixteen bytes of a row of y or out; n: elements that the row has from p on.
template <typename T> struct Piece;
template <> struct Piece<uint16_t> {
  static constexpr int N = 8;
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= N) {
      v = *reinterpret_cast<const u32x4_2l*>(p);
    } else {
      v = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  __device__ __forceinline__ void store(uint16_t* p, int n) const {
    if (n >= N) {
      *reinterpret_cast<u32x4_2l*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
  }
  __device__ __forceinline__ void add(int i, f32x4l d) {  // elements 4i .. 4i + 3
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t w = v[2 * i + e];
      const f32x2l f = {__uint_as_float(w << 16) + d[2 * e], __uint_as_float(w & 0xFFFF0000u) + d[2 * e + 1]};
      v[2 * i + e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2l));
    }
  }
};
template <> struct Piece<float> {
  static constexpr int N = 4;
  u32x4 v;
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= N) {
      v = *reinterpret_cast<const u32x4_4l*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = i < n ? __float_as_uint(p[i]) : 0u;
    }
  }
  __device__ __forceinline__ void store(float* p, int n) const {
    if (n >= N) {
      *reinterpret_cast<u32x4_4l*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) p[i] = __uint_as_float(v[i]);
    }
  }
  __device__ __forceinline__ void add(int, f32x4l d) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + d[e]);
  }
};

// out of a tile's rows, 64 columns a wave and step, as four products of 16
// columns.  Which columns those are is free: row m of product i is column
//   4 E (i / Q) + E (m / 4) + 4 (i % Q) + m % 4,  E elements of 16 bytes, Q = E / 4,
// so that a lane's results are whole pieces of 16 bytes of one row, and the four
// lanes that share a row load and store 64 bytes together.
template <typename T, int MT, int RS, bool Y>
__global__ __launch_bounds__(256) void k_lora_out(LoraArgs p) {
  constexpr int TM = 16 * MT, RP = 32 * RS, TERMS = sizeof(T) == 2 ? 2 : 3, PAD = RP + 8;
  constexpr int E = Piece<T>::N, Q = E / 4, P = 4 / Q;  // P pieces of a lane
  __shared__ __attribute__((aligned(16))) uint16_t s_u[TERMS][TM][PAD];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const LoraTile t = lora_tile<TM>(p, tile);
  if (t.n == 0) return;
  const int64_t first = (int64_t)part * p.iters * 256 + wave * 64;
  const T* y = static_cast<const T*>(p.y);
  T* out = static_cast<T*>(p.out);
  if (t.a < 0) {  // no adapter: y's rows
    if (Y && y == out) return;
    const int64_t from = (int64_t)part * p.iters * 256, to = min(p.N, from + (int64_t)p.iters * 256);
    for (int row = wave; row < t.n; row += 4)
      for (int64_t n = from + lane * E; n < to; n += 64 * E) {
        const int left = (int)min((int64_t)E, p.N - n);
        Piece<T> o;
        if (Y) o.load(y + (t.r0 + row) * p.ldy + n, left);
        else o.v = u32x4{0, 0, 0, 0};
        o.store(out + (t.r0 + row) * p.ldo + n, left);
      }
    return;
  }
  struct Step {
    Piece<T> o[MT][P];
    u32x4 b[4];
  };
  // Loads without conditions, so that none waits for another: of columns, ranks
  // and rows that are not there, some that are.
  auto load_b = [&](Step& f, int64_t n0, int s) {  // B's for ranks 32 s ..
    const int r = 32 * s + 8 * g < p.rank ? 32 * s + 8 * g : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t n = min(n0 + 4 * E * (i / Q) + E * (c >> 2) + 4 * (i % Q) + (c & 3), p.N - 1);
      f.b[i] = *reinterpret_cast<const u32x4*>(p.b + ((int64_t)t.a * p.N + n) * p.rank + r);
    }
  };
  auto load = [&](Step& f, int64_t n0) {  // (whole steps: columns n0 .. n0 + 63 are there)
    load_b(f, n0, 0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (Y) f.o[m][j].load(y + (t.r0 + min(16 * m + c, t.n - 1)) * p.ldy + n0 + 4 * E * j + E * g, E);
        else f.o[m][j].v = u32x4{0, 0, 0, 0};
      }
  };
  auto no_tail = [&](Step& f, int s) {  // ranks that are not there
    if (32 * s + 32 > p.rank) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (32 * s + 8 * g >= p.rank) f.b[i] = u32x4{0, 0, 0, 0};
    }
  };
  auto zero = [](f32x4l (&acc)[MT][4]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = {0.0f, 0.0f, 0.0f, 0.0f};
  };
  auto term = [&](Step& f, int s, int e, f32x4l (&acc)[MT][4]) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const u32x4 fu = *reinterpret_cast<const u32x4*>(&s_u[e][16 * m + c][32 * s + 8 * g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = product(f.b[i], fu, acc[m][i]);
    }
  };
  auto add = [&](Step& f, int64_t n0) {
    f32x4l acc[MT][4];
    zero(acc);
#pragma unroll
    for (int s = 0; s < RS; ++s) {
      if (s > 0) load_b(f, n0, s);
      no_tail(f, s);
#pragma unroll
      for (int e = 0; e < TERMS; ++e) term(f, s, e, acc);
    }
    // An infinite element of B times a lower term that is 0, or of the other sign,
    // has made NaN of an infinite result.  Where a sum is infinite or NaN (`any` then
    // is; two large ones make it so too, and come out again), the lower terms
    // take B's finite elements alone.
    float any = 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        any = __builtin_fmaf(acc[m][i][0], acc[m][i][1], any);
        any = __builtin_fmaf(acc[m][i][2], acc[m][i][3], any);
      }
    if (__any(!(fabsf(any) < INFINITY))) {
      int64_t again = n0;  // (its own addresses: shared ones would be held in registers)
      asm volatile("" : "+s"(again));
      zero(acc);
#pragma unroll 1
      for (int s = 0; s < RS; ++s) {
        load_b(f, again, s);
        no_tail(f, s);
        term(f, s, 0, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) f.b[i] = finite_of(f.b[i]);
#pragma unroll 1
        for (int e = 1; e < TERMS; ++e) term(f, s, e, acc);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) f.o[m][i / Q].add(i % Q, acc[m][i]);
  };
  auto finish = [&](Step& f, int64_t n0) {
    add(f, n0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (16 * m + c < t.n) {
#pragma unroll
        for (int j = 0; j < P; ++j) f.o[m][j].store(out + (t.r0 + 16 * m + c) * p.ldo + n0 + 4 * E * j + E * g, E);
      }
  };
  // this wave's whole steps, and the columns after the last one
  const int64_t end = min(p.N, first + (int64_t)p.iters * 256);
  const int64_t whole = first + 64 <= end ? (end - 64 - first) / 256 + 1 : 0, last = first + whole * 256;
  Step f0, f1;
  if (whole > 0) load(f0, first);  // (on its way while u is split)
  // u as BF16 terms: a thread four ranks of a row
  const float s = p.scale ? p.scale[t.a] : 1.0f;
  for (int i = threadIdx.x; i < TM * RP / 4; i += 256) {
    const int row = i / (RP / 4), r = i % (RP / 4) * 4;
    f32x4l v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (row < t.n && r < p.rank) {
      const float* u = p.u + (t.r0 + row) * p.ur + r;
      for (int k = 0; k < p.splits; k += 4) {  // four splits' loads together
        f32x4l w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = *reinterpret_cast<const f32x4l*>(u + min(k + j, p.splits - 1) * p.rows * p.ur);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k + j < p.splits) v += w[j];
      }
      v *= s;
    }
#pragma unroll
    for (int e = 0; e < TERMS; ++e) {
      f32x4l t = v;
      if (e == 0) {  // (finite values that would be rounded to infinity: the largest BF16)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (fabsf(v[j]) < INFINITY) t[j] = __builtin_amdgcn_fmed3f(v[j], -BF16_MAX, BF16_MAX);
      }
      const f32x2l lo = {t[0], t[1]}, hi = {t[2], t[3]};
      const u32x2 w = {__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2l)),
                       __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2l))};
      *reinterpret_cast<u32x2*>(&s_u[e][row][r]) = w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // (an infinity is one term)
        const float term = __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
        v[j] = fabsf(term) == INFINITY ? 0.0f : v[j] - term;
      }
    }
  }
  __syncthreads();
  // a step's loads on their way while the one before is finished (after the last
  // its own again)
  for (int64_t i = 0; i < whole; i += 2) {
    const int64_t n0 = first + i * 256;
    load(f1, first + min(i + 1, whole - 1) * 256);
    finish(f0, n0);
    if (i + 1 >= whole) break;
    load(f0, first + min(i + 2, whole - 1) * 256);
    finish(f1, n0 + 256);
  }
  if (last >= end) return;
  load_b(f0, last, 0);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int64_t at = last + 4 * E * j + E * g;
      f0.o[m][j].v = u32x4{0, 0, 0, 0};
      if (Y && 16 * m + c < t.n && at < p.N)
        f0.o[m][j].load(y + (t.r0 + 16 * m + c) * p.ldy + at, (int)min((int64_t)E, p.N - at));
    }
  add(f0, last);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int64_t at = last + 4 * E * j + E * g;
      if (16 * m + c < t.n && at < p.N)
        f0.o[m][j].store(out + (t.r0 + 16 * m + c) * p.ldo + at, (int)min((int64_t)E, p.N - at));
    }
}

// How a call is split, from host numbers only (each request may leave a tile that
// is not full, and so may the rows of none).  Its rules, with what the other choice
// takes (us, both sides without the look at a step's sums; prompt: 8192 rows of 11 requests, rank 32, K 4096, N 14336, BF16; step:
// 64 requests of one row, rank 16, the same K and N):
//   many    tiles of 64 rows for u (32 for ranks above 64: 26, by 64 37) and 32 for out
//           from 1024 rows and 32 a request on, else 16: prompt u 21.6, by 32 rows 24.9; out
//           109, by 64 rows 113; 121 rows of rank 128 5.8 + 7.0, by many 10.3 + 13.0
//   splits  of K, for 512 workgroups, each 1024 of K at least: prompt 22, for 256 28
//   iters   steps of a workgroup of out: prompt 1, 2, 3, 4, 6: 154, 123, 115, 109, 121; at
//           2489 rows and 9186 columns of F32 57, 49, 46, 45, 44; fewer where 256
//           workgroups would not be reached (3082 rows, 671 columns: 2 12.6, 3 18.0).  Small
//           tiles: for 1024 workgroups (step: for 512, 1024, 2048 8.4, 8.5, 10.3).  A tile's
//           workgroups follow one another: by tiles first 124 (prompt, 64 rows)
struct LoraPlan {
  bool many;  // rows enough for tiles of several products
  int rt, rs, splits, iters, parts;
  int64_t u_tiles, out_tiles, chunk;
};

LoraPlan lora_plan(int64_t rows, int G, int rank, int64_t K, int64_t N) {
  LoraPlan p;
  p.many = rows >= 32 * (int64_t)G && rows >= 1024;
  p.rt = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
  p.rs = p.rt <= 2 ? 1 : p.rt / 2;
  auto tiles = [&](int tm) {
    const int64_t full = rows / tm + (int64_t)G + 1;
    return full < rows ? full : rows;
  };
  p.u_tiles = tiles(16 * (!p.many ? 1 : p.rt == 8 ? U_MT_128 : U_MT));
  p.out_tiles = tiles(16 * (p.many ? OUT_MT : 1));
  int64_t s = (512 + p.u_tiles - 1) / p.u_tiles;
  const int64_t most = (K + 1023) / 1024;
  s = s < most ? s : most;
  p.chunk = ((K + s - 1) / s + 127) / 128 * 128;
  p.splits = (int)((K + p.chunk - 1) / p.chunk);
  const int64_t steps = (N + 255) / 256, want = p.many ? 256 : 1024;
  int64_t it = (p.out_tiles * steps + want - 1) / want;
  if (p.many && it > 4) it = 4;
  p.iters = (int)(it < steps ? it : steps);
  p.parts = (int)((steps + p.iters - 1) / p.iters);
  return p;
}

template <int MT>
void launch_u(const LoraArgs& p, const LoraPlan& pl, hipStream_t stream) {
  const dim3 grid((unsigned)pl.u_tiles, (unsigned)pl.splits);
  if (pl.rt == 1) hipLaunchKernelGGL((k_lora_u<MT, 1>), grid, dim3(256), 0, stream, p);
  else if (pl.rt == 2) hipLaunchKernelGGL((k_lora_u<MT, 2>), grid, dim3(256), 0, stream, p);
  else if (pl.rt == 4) hipLaunchKernelGGL((k_lora_u<MT, 4>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((k_lora_u<(MT == U_MT ? U_MT_128 : MT), 8>), grid, dim3(256), 0, stream, p);
}

template <typename T, int MT, bool Y>
void launch_out(const LoraArgs& p, const LoraPlan& pl, hipStream_t stream) {
  const dim3 grid((unsigned)(pl.out_tiles * pl.parts));
  if (pl.rs == 1) hipLaunchKernelGGL((k_lora_out<T, MT, 1, Y>), grid, dim3(256), 0, stream, p);
  else if (pl.rs == 2) hipLaunchKernelGGL((k_lora_out<T, MT, 2, Y>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((k_lora_out<T, MT, 4, Y>), grid, dim3(256), 0, stream, p);
}

template <typename T>
void launch_type(const LoraArgs& p, const LoraPlan& pl, hipStream_t stream) {
  if (pl.many) {
    if (p.y) launch_out<T, OUT_MT, true>(p, pl, stream);
    else launch_out<T, OUT_MT, false>(p, pl, stream);
  } else {
    if (p.y) launch_out<T, 1, true>(p, pl, stream);
    else launch_out<T, 1, false>(p, pl, stream);
  }
}

}  // namespace

size_t lora_workspace_bytes(int64_t rows, int G, int rank, int64_t K, int64_t N) {
  const LoraPlan pl = lora_plan(rows, G, rank, K, N);
  return (size_t)pl.splits * (size_t)rows * (size_t)(pl.rt * 16) * 4;
}

void launch_lora(int f32, const uint16_t* x, int64_t ldx, const uint16_t* a, const uint16_t* b, const float* scale,
                 int adapters, int rank, const int32_t* off, const int32_t* adapter, int G, int64_t rows, int64_t K,
                 int64_t N, const void* y, int64_t ldy, void* out, int64_t ldo, void* ws, hipStream_t stream) {
  const LoraPlan pl = lora_plan(rows, G, rank, K, N);
  const LoraArgs p = {x, ldx, a, b, scale, adapters, rank, off, adapter, G, rows, K, N, y, ldy, out, ldo,
                      static_cast<float*>(ws), pl.rt * 16, pl.splits, pl.chunk, pl.iters, pl.parts};
  if (pl.many) launch_u<U_MT>(p, pl, stream);
  else launch_u<1>(p, pl, stream);
  if (f32) launch_type<float>(p, pl, stream);
  else launch_type<uint16_t>(p, pl, stream);
}

}  // namespace fp4q
