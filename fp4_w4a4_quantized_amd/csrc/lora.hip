// lora.hip -- low-rank adapters of many requests beside a shared projection
// (defined in include/fp4q.h): for the rows of each request,
//   out = y + s (x A^T) B^T   with its adapter's A [rank, K], B [N, rank].
//
// Bound by HBM: y is read and written once, x read once (prompts), or the
// adapters' A and B, which a request of one token reads whole (decode).  Two
// kernels: u = x A^T with K split over the waves and, where there are few rows,
// over workgroups (partial sums in F32, added in order by the second kernel);
// then out, each workgroup some columns of a tile of rows.
//
// Products are 16x16x32 on BF16.  x, A and B enter as they are; u enters the
// second product as two BF16 terms (u but for 2^-17) where out is BF16, as three
// (2^-25) where it is F32: one term, 2^-9, would be as large as out's own rounding.
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
  int iters;           // 256-column steps of a workgroup
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
    int r0 = 0, r1 = 0, id = -1;
    if (g <= p.G) {
      r0 = min(max(p.off[g], 0), rows);
      r1 = g < p.G ? min(max(p.off[g + 1], r0), rows) : rows;
      if (g < p.G) id = p.adapter[g];
    }
    const int mine = (r1 - r0 + TM - 1) / TM;
    const int to = before + sum_to_lane(mine), first = to - mine;  // of this request's tiles
    const uint64_t hit = __ballot(tile >= first && tile < to);
    if (hit) {
      const int at = __ffsll((unsigned long long)hit) - 1;
      auto of = [&](int v) { return __builtin_amdgcn_readlane(v, at); };
      const int from = of(r0) + (tile - of(first)) * TM;
      t.r0 = from;
      t.n = min(TM, of(r1) - from);
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
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const LoraTile t = lora_tile<TM>(p, blockIdx.x);
  if (t.n == 0 || t.a < 0) return;
  const int64_t k0 = blockIdx.y * p.chunk, k1 = min(p.K, k0 + p.chunk);
  const uint16_t* a[RT];
  const uint16_t* x[MT];
  bool a_on[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    a_on[i] = 16 * i + c < p.rank;
    a[i] = p.a + ((int64_t)t.a * p.rank + (a_on[i] ? 16 * i + c : 0)) * p.K + 8 * g;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) x[i] = p.x + (t.r0 + min(16 * i + c, t.n - 1)) * p.ldx + 8 * g;
  f32x4l acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[m][i] = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = MT * RT >= 32 ? 1 : MT * RT >= 8 ? 2 : 4;  // steps of 32 along K that are loaded together
  struct Batch {
    u32x4 a[U][RT], x[U][MT];
  };
  auto load = [&](Batch& f, int64_t k) {
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const bool in = k + 32 * s + 8 * g < k1;  // (K and a split's end are multiples of 8)
#pragma unroll
      for (int i = 0; i < RT; ++i)
        f.a[s][i] = in && a_on[i] ? *reinterpret_cast<const u32x4*>(a[i] + k + 32 * s) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int m = 0; m < MT; ++m)
        f.x[s][m] = in ? *reinterpret_cast<const u32x4*>(x[m] + k + 32 * s) : u32x4{0, 0, 0, 0};
    }
  };
  auto multiply = [&](const Batch& f) {
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
    multiply(f0);
    if (k + STRIDE >= k1) break;
    if (k + 2 * STRIDE < k1) load(f0, k + 2 * STRIDE);
    multiply(f1);
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

// Sixteen neighbouring elements of a row of y or out, from column n0 on.
template <typename T> struct Sixteen;
template <> struct Sixteen<uint16_t> {
  u32x4 v[2];
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= 16) {
      v[0] = *reinterpret_cast<const u32x4_2l*>(p);
      v[1] = *reinterpret_cast<const u32x4_2l*>(p + 8);
    } else {
      v[0] = v[1] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) v[i >> 3][(i >> 1) & 3] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  __device__ __forceinline__ void store(uint16_t* p, int n) const {
    if (n >= 16) {
      *reinterpret_cast<u32x4_2l*>(p) = v[0];
      *reinterpret_cast<u32x4_2l*>(p + 8) = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) p[i] = (uint16_t)(v[i >> 3][(i >> 1) & 3] >> (16 * (i & 1)));
    }
  }
  __device__ __forceinline__ void add(int i, f32x4l d) {  // elements 4i .. 4i + 3
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t w = v[i >> 1][2 * (i & 1) + e];
      const f32x2l f = {__uint_as_float(w << 16) + d[2 * e], __uint_as_float(w & 0xFFFF0000u) + d[2 * e + 1]};
      v[i >> 1][2 * (i & 1) + e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2l));
    }
  }
};
template <> struct Sixteen<float> {
  u32x4 v[4];
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const u32x4_4l*>(p + 4 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i >> 2][i & 3] = i < n ? __float_as_uint(p[i]) : 0u;
    }
  }
  __device__ __forceinline__ void store(float* p, int n) const {
    if (n >= 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4_4l*>(p + 4 * i) = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) p[i] = __uint_as_float(v[i >> 2][i & 3]);
    }
  }
  __device__ __forceinline__ void add(int i, f32x4l d) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i][e] = __float_as_uint(__uint_as_float(v[i][e]) + d[e]);
  }
};

// out of a tile's rows, 64 columns a wave and step.  Row m of product i is column
// 16 (m / 4) + 4 i + m % 4 of the 64, so that a lane's four products are 16
// neighbouring columns of one row, and 16 lanes' loads of y whole lines.
template <typename T, int MT, int RS>
__global__ __launch_bounds__(256) void k_lora_out(LoraArgs p) {
  constexpr int TM = 16 * MT, RP = 32 * RS, TERMS = sizeof(T) == 2 ? 2 : 3, PAD = RP + 8;
  __shared__ __attribute__((aligned(16))) uint16_t s_u[TERMS][TM][PAD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const LoraTile t = lora_tile<TM>(p, blockIdx.x);
  if (t.n == 0 || (t.a < 0 && p.y == p.out)) return;
  const int64_t first = (int64_t)blockIdx.y * p.iters * 256 + wave * 64;
  const T* y = static_cast<const T*>(p.y);
  Sixteen<T> o[MT];
  u32x4 fb[4];
  auto load_b = [&](int64_t n0, int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t n = n0 + 16 * (c >> 2) + 4 * i + (c & 3);
      fb[i] = t.a >= 0 && n < p.N && 32 * s + 8 * g < p.rank
                  ? *reinterpret_cast<const u32x4*>(p.b + ((int64_t)t.a * p.N + n) * p.rank + 32 * s + 8 * g)
                  : u32x4{0, 0, 0, 0};
    }
  };
  auto load = [&](int64_t n0) {  // y's part, and B's for the first ranks
    const int64_t at = n0 + 16 * g;
    const int left = (int)min((int64_t)16, p.N - at);  // (below 1: none of this lane's)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = 16 * m + c;
      if (y && row < t.n && left > 0) {
        o[m].load(y + (t.r0 + row) * p.ldy + at, left);
      } else {
#pragma unroll
        for (auto& w : o[m].v) w = u32x4{0, 0, 0, 0};
      }
    }
    load_b(n0, 0);
  };
  load(first);  // (on its way while u is split)
  if (t.a >= 0) {
    // u as BF16 terms: a thread four ranks of a row
    const float s = p.scale ? p.scale[t.a] : 1.0f;
    for (int i = threadIdx.x; i < TM * RP / 4; i += 256) {
      const int row = i / (RP / 4), r = i % (RP / 4) * 4;
      f32x4l v = {0.0f, 0.0f, 0.0f, 0.0f};
      if (row < t.n && r < p.rank) {
        const float* u = p.u + (t.r0 + row) * p.ur + r;
        for (int k = 0; k < p.splits; ++k) v += *reinterpret_cast<const f32x4l*>(u + k * p.rows * p.ur);
        v *= s;
      }
#pragma unroll
      for (int e = 0; e < TERMS; ++e) {
        const f32x2l lo = {v[0], v[1]}, hi = {v[2], v[3]};
        const u32x2 w = {__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2l)),
                         __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2l))};
        *reinterpret_cast<u32x2*>(&s_u[e][row][r]) = w;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] -= __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
      }
    }
    __syncthreads();
  }
  T* out = static_cast<T*>(p.out);
  for (int it = 0; it < p.iters; ++it) {
    const int64_t n0 = first + it * 256;
    if (n0 >= p.N) break;
    if (it > 0) load(n0);
    if (t.a >= 0) {
      f32x4l acc[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        if (s > 0) load_b(n0, s);
#pragma unroll
        for (int e = 0; e < TERMS; ++e)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const u32x4 fu = *reinterpret_cast<const u32x4*>(&s_u[e][16 * m + c][32 * s + 8 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i] = product(fb[i], fu, acc[m][i]);
          }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m].add(i, acc[m][i]);
    }
    const int left = (int)min((int64_t)16, p.N - (n0 + 16 * g));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = 16 * m + c;
      if (row < t.n && left > 0) o[m].store(out + (t.r0 + row) * p.ldo + n0 + 16 * g, left);
    }
  }
}

// How a call is split, from host numbers only: rows of a tile, tiles at most
// (every request may leave one that is not full, and so may the rows of none),
// splits of K, columns of a workgroup.
struct LoraPlan {
  int mt, rt, rs, splits, iters;
  int64_t tiles, chunk;
};

LoraPlan lora_plan(int64_t rows, int G, int rank, int64_t K, int64_t N) {
  LoraPlan p;
  p.mt = rows >= 32 * (int64_t)G ? 4 : 1;
  p.rt = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
  p.rs = p.rt <= 2 ? 1 : p.rt / 2;
  const int tm = 16 * p.mt;
  const int64_t full = rows / tm + (int64_t)G + 1;
  p.tiles = full < rows ? full : rows;
  int64_t s = (512 + p.tiles - 1) / p.tiles;
  const int64_t most = (K + 1023) / 1024;
  s = s < most ? s : most;
  p.chunk = ((K + s - 1) / s + 127) / 128 * 128;
  p.splits = (int)((K + p.chunk - 1) / p.chunk);
  const int64_t steps = (N + 255) / 256;
  const int64_t it = (p.tiles * steps + 2047) / 2048;
  p.iters = (int)(it < 1 ? 1 : it < steps ? it : steps);
  return p;
}

template <int MT>
void launch_u(const LoraArgs& p, const LoraPlan& pl, hipStream_t stream) {
  const dim3 grid((unsigned)pl.tiles, (unsigned)pl.splits);
  if (pl.rt == 1) hipLaunchKernelGGL((k_lora_u<MT, 1>), grid, dim3(256), 0, stream, p);
  else if (pl.rt == 2) hipLaunchKernelGGL((k_lora_u<MT, 2>), grid, dim3(256), 0, stream, p);
  else if (pl.rt == 4) hipLaunchKernelGGL((k_lora_u<MT, 4>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((k_lora_u<MT, 8>), grid, dim3(256), 0, stream, p);
}

template <typename T, int MT>
void launch_out(const LoraArgs& p, const LoraPlan& pl, hipStream_t stream) {
  const int64_t steps = (p.N + 255) / 256;
  const dim3 grid((unsigned)pl.tiles, (unsigned)((steps + pl.iters - 1) / pl.iters));
  if (pl.rs == 1) hipLaunchKernelGGL((k_lora_out<T, MT, 1>), grid, dim3(256), 0, stream, p);
  else if (pl.rs == 2) hipLaunchKernelGGL((k_lora_out<T, MT, 2>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((k_lora_out<T, MT, 4>), grid, dim3(256), 0, stream, p);
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
                      static_cast<float*>(ws), pl.rt * 16, pl.splits, pl.chunk, pl.iters};
  if (pl.mt == 4) launch_u<4>(p, pl, stream);
  else launch_u<1>(p, pl, stream);
  if (f32) {
    if (pl.mt == 4) launch_out<float, 4>(p, pl, stream);
    else launch_out<float, 1>(p, pl, stream);
  } else {
    if (pl.mt == 4) launch_out<uint16_t, 4>(p, pl, stream);
    else launch_out<uint16_t, 1>(p, pl, stream);
  }
}

}  // namespace fp4q
