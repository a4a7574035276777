// norm.hip -- the root-mean-square norm of a residual stream (defined in
// include/fp4q.h): per row
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r weight,
// with y written, or quantized into the operand of the product behind it
// (NVFP4, MXFP4, MXFP8) with the residual of selected channels, its gradient,
// and the values that an operand stands for.
//
// All of it is bound by HBM: x and the residual are read once, h, y or the codes
// written once, with a row in the registers of one, four or eight waves in
// between.  NVFP4's own tensor scale needs every row's y before the first code: a
// first pass writes h, each row's r and the workgroups' maxima, a second reads h
// again.  8192 x 4096 BF16 with a residual: the first 35 us (201 MB, 5.7 TB/s), the
// second 26.2 (17 vector instructions an element: 18 us); with a given scale, in one
// pass, 47.1 and MXFP4 45.6 (222 MB, 4.7 and 4.8 TB/s); MXFP8 in one pass 41.5
// (236 MB, 5.7 TB/s); 4099 rows of y 24.3 and of the gradient 29 (134 MB, 5.5 and 4.6),
// the sum of d_weight 6.5.
//
// The sum of squares, r and y are 64-bit: y then is the definition's F32 value
// but in 2^-28 of the cases, and the BF16 value and code made of it with it; a y
// of 32-bit steps lies an ulp apart often enough that codes next to a border
// differ.  It costs one conversion each way and one product an element.
#include "fp4q_device.h"
#include "fp4q_internal.h"

namespace fp4q {

namespace {

typedef float f32x2n __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2n __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2n __attribute__((ext_vector_type(2)));
// Sixteen bytes at any element's address (rows of odd strides).
typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));

struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* res;  // or null
  int64_t ldr;
  void* h;          // null: no residual (h is x)
  int64_t ldh;
  const void* w;
  int w_f32;
  double eps;
  int64_t rows;
  int cols;
  void* y;          // or null
  int64_t ldy;
  int y_f32;
  float* rstd;      // or null
  // quantized output
  uint8_t* q;
  uint8_t* scales;
  float* tscale;    // NVFP4: given, or written from the maxima
  int n_max;        // maxima of the first pass
  float* maxima;
  double* r64;      // the rows' r, first pass to second
  bool tiled;
  const int32_t* chan;
  int n_chan;
  uint16_t* resid;
  int64_t groups;   // groups of rows: one to a workgroup at a time
};

enum { EMIT_Y, EMIT_MAX, EMIT_NVFP4, EMIT_MXFP4, EMIT_MXFP8 };

constexpr int CH = 8;  // elements of a lane's chunk
// Workgroups of a pass; further rows in turn: four on each CU, so that a row's loads are
// ahead of its work.  us of NVFP4's two passes for 512, 1024, 2048:
// 8192 x 4096 65.8, 60.3, 62.0; 16384 x 1024 40.0, 35.7, 37.2; 8192 x 2048 48.2, 36.8,
// 38.2 (MXFP8 of 4096 x 8192 loses: 52.1, 53.5, 48.3).
constexpr int MAX_WGS = 1024;

// Eight elements as they stand in memory.
template <typename T> struct Raw;
template <> struct Raw<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float((i & 1) ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
  }
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= CH) {
      v = *reinterpret_cast<const u32x4_2*>(p);
    } else {
      v = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (i < n) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  __device__ __forceinline__ void store(uint16_t* p, int n) const {
    if (n >= CH) {
      *reinterpret_cast<u32x4_2*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (i < n) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
  }
  __device__ __forceinline__ void set(const float (&f)[CH]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2n t = {f[2 * i], f[2 * i + 1]};
      v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(t, bf16x2n));
    }
  }
};
template <> struct Raw<float> {
  u32x4 v[2];
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(v[i >> 2][i & 3]); }
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= CH) {
      v[0] = *reinterpret_cast<const u32x4_4*>(p);
      v[1] = *reinterpret_cast<const u32x4_4*>(p + 4);
    } else {
      v[0] = v[1] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (i < n) v[i >> 2][i & 3] = __float_as_uint(p[i]);
    }
  }
  __device__ __forceinline__ void store(float* p, int n) const {
    if (n >= CH) {
      *reinterpret_cast<u32x4_4*>(p) = v[0];
      *reinterpret_cast<u32x4_4*>(p + 4) = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (i < n) p[i] = at(i);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[CH]) {
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i >> 2][i & 3] = __float_as_uint(f[i]);
  }
};

// Elements that a row of WPR waves with N chunks a lane has room for.
constexpr int room(int wpr, int n) { return wpr * 64 * CH * n; }

__device__ __forceinline__ void load_any(const void* p, int64_t at, int f32, int n, float (&f)[CH]) {
  if (f32) {
    Raw<float> r;
    r.load(static_cast<const float*>(p) + at, n);
#pragma unroll
    for (int i = 0; i < CH; ++i) f[i] = r.at(i);
  } else {
    Raw<uint16_t> r;
    r.load(static_cast<const uint16_t*>(p) + at, n);
#pragma unroll
    for (int i = 0; i < CH; ++i) f[i] = r.at(i);
  }
}

__device__ __forceinline__ void store_any(void* p, int64_t at, int f32, int n, const float (&f)[CH]) {
  if (f32) {
    Raw<float> r;
    r.set(f);
    r.store(static_cast<float*>(p) + at, n);
  } else {
    Raw<uint16_t> r;
    r.set(f);
    r.store(static_cast<uint16_t*>(p) + at, n);
  }
}

__device__ __forceinline__ uint32_t max_bits(const Raw<uint16_t>& r) {
  u16x2n m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2n, r.v[i] & 0x7FFF7FFFu));
  return max((uint32_t)m[0], (uint32_t)m[1]);
}

// The largest of v over the N (2 or 4) lanes whose chunks make up a block.
template <int N>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  if (N == 4) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
  return v;
}

// The tensor scale t as the NVFP4 encoder takes it.  Where it and every divisor
// scale * t lie within quot_rn's range (all but the most extreme t), reciprocals
// stand in a table by scale code and no division is left; else rt is 0.
struct TensorScale {
  float t, rt;
  const float* reciprocal;  // LDS: RN(1 / (scale t)) by code, 0 for code 0
};

// quot_rn of a BF16 x: one correction is enough (it gives the IEEE quotient for each
// of the 2^7 mantissas of x by each of the 2^23 of d).
__device__ __forceinline__ float quot_bf16(float x, float d, float y) {
  const float q = x * y;
  return __builtin_fmaf(-__builtin_fmaf(q, d, -x), y, q);
}

// A chunk of y (BF16) as codes: FP4's in w[0], MXFP8's in w[0], w[1]; returns the
// block's scale code.  FAR: a given tensor scale, whose blocks may lie far past
// what it can hold (their operands are held within 8 divisors: beyond that every
// quotient gives the largest code).
template <int EMIT, bool FAR>
__device__ __forceinline__ uint32_t encode(const Raw<uint16_t>& y, uint32_t amax_bits, const TensorScale& ts,
                                           uint32_t (&w)[2]) {
  const float amax = bf16_to_f32(amax_bits);
  float v[CH];
  if constexpr (EMIT == EMIT_NVFP4) {
    if (ts.rt != 0.0f) {
      // amax / 6: one correction of amax RN(1/6) is the IEEE quotient for every BF16 amax
      const float q = amax * (1.0f / 6.0f);
      const float a6 = __builtin_fmaf(__builtin_fmaf(-q, 6.0f, amax), 1.0f / 6.0f, q);
      const uint32_t sb = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fminf(quot_rn(a6, ts.t, ts.rt), 448.0f), 0.0f,
                                                                    0, false) & 0x7Fu;
      const float d = e4m3_value(sb) * ts.t, rd = ts.reciprocal[sb];
#pragma unroll
      for (int i = 0; i < CH; ++i)
        v[i] = quot_bf16(FAR ? __builtin_amdgcn_fmed3f(y.at(i), -8.0f * d, 8.0f * d) : y.at(i), d, rd);
      w[0] = e2m1_pack8(v);
      return sb;
    }
    const uint32_t sb = e4m3_encode((amax / 6.0f) / ts.t);
    const float d = e4m3_value(sb) * ts.t;
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] = d > 0.0f ? y.at(i) / d : 0.0f * y.at(i);
    w[0] = e2m1_pack8(v);
    return sb & 0xFFu;
  } else if constexpr (EMIT == EMIT_MXFP4) {
    const int e8 = mx_exponent(amax);
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] = y.at(i);
    w[0] = e2m1_pack8(v, __uint_as_float((uint32_t)(e8 + 127) << 23));
    return (uint32_t)(e8 + 127);
  } else {
    const int e8 = mx8_exponent(amax);
    // times 2^-e, exact where it matters (what underflows is below half the
    // smallest step)
    const float s = exp2i(-e8);
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] = y.at(i) * s;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t u = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], (int)u, true);
    }
    return (uint32_t)(e8 + 127);
  }
}

// Sums and maxima over a wave by vector moves: within four lanes, eight, sixteen
// (whose lanes then hold the same), and the lanes 16 and 32 apart.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

template <typename T, typename F>
__device__ __forceinline__ T over_wave(T v, F join) {
  constexpr int N = sizeof(T) / 4;
  union U {
    T t;
    uint32_t w[N];
  };
#define FP4Q_STEP(MOVE)                                    \
  {                                                        \
    U a, b;                                                \
    a.t = v;                                               \
    _Pragma("unroll") for (int i = 0; i < N; ++i) b.w[i] = MOVE(a.w[i]); \
    v = join(a.t, b.t);                                    \
  }
  FP4Q_STEP(moved<0xB1>)
  FP4Q_STEP(moved<0x4E>)
  FP4Q_STEP(moved<0x141>)
  FP4Q_STEP(moved<0x140>)
#undef FP4Q_STEP
#define FP4Q_SWAP(SWAP)                                                                        \
  {                                                                                            \
    U a, p, q;                                                                                 \
    a.t = v;                                                                                   \
    _Pragma("unroll") for (int i = 0; i < N; ++i) {                                            \
      const u32x2 r = __builtin_bit_cast(u32x2, SWAP(a.w[i], a.w[i], false, false));           \
      p.w[i] = r[0];                                                                           \
      q.w[i] = r[1];                                                                           \
    }                                                                                          \
    v = join(p.t, q.t);                                                                        \
  }
  FP4Q_SWAP(__builtin_amdgcn_permlane16_swap)
  FP4Q_SWAP(__builtin_amdgcn_permlane32_swap)
#undef FP4Q_SWAP
  return v;
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
  return over_wave(v, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return over_wave(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// The group of rows that workgroup g takes.  Workgroups go to the eight XCDs in
// turn; the 16 rows of a tiled block of codes are written by one of them (each
// writes 16 bytes of a line, which meet in its cache).
__device__ __forceinline__ int64_t row_group(int64_t g, int64_t groups, int per16, bool tiled) {
  const int64_t all = 8 * per16, base = g / all * all;
  if (!tiled || base + all > groups) return g;
  const int i = (int)(g - base);
  return base + (i & 7) * per16 + (i >> 3);
}

// WPR: waves of a row (a workgroup of four rows, or one); N: chunks of a lane at
// most.  SECOND: r and h are given (the second pass of NVFP4's own tensor scale).
template <typename T, int WPR, int N, int EMIT, bool SECOND>
__global__ __launch_bounds__(WPR == 8 ? 512 : 256) void k_norm(NormArgs p) {
  constexpr int ROWS = WPR == 1 ? 4 : 1, WAVES = WPR * ROWS;
  constexpr bool QUANT = EMIT >= EMIT_NVFP4;
  // per row, for the selected channels: y, codes and scale codes
  extern __shared__ __attribute__((aligned(16))) uint8_t s_rows[];
  __shared__ double s_sum[2][WAVES];
  __shared__ uint32_t s_max[WAVES];
  __shared__ float s_rec[EMIT == EMIT_NVFP4 ? 128 : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = WPR == 1 ? 0 : wave;
  const int nc = (p.cols + WPR * 64 * CH - 1) / (WPR * 64 * CH);
  const int col0 = (sub * 64 + lane) * CH;  // of chunk 0; chunk c: WPR * 512 c further
  uint8_t* const mine = s_rows + (WPR == 1 ? wave * 4 * p.cols : 0);
  uint16_t* const ys = reinterpret_cast<uint16_t*>(mine);
  uint32_t* const codes = reinterpret_cast<uint32_t*>(mine + 2 * p.cols);
  uint8_t* const scs = mine + 2 * p.cols + p.cols / 2;
  // whole chunks where the columns are a multiple of 8
  auto left = [&](int col) { return EMIT == EMIT_Y ? p.cols - col : CH; };
  // a row's x (or h) and residual
  struct In {
    Raw<T> x[N], res[N];
    double r;
  };
  const T* const xs = static_cast<const T*>(SECOND && p.h ? p.h : p.x);
  const int64_t ldx = SECOND && p.h ? p.ldh : p.ldx;
  auto row_of = [&](int64_t g) { return row_group(g, p.groups, 16 / ROWS, p.tiled) * ROWS + (WPR == 1 ? wave : 0); };
  auto load = [&](In& in, int64_t row) {
    if (WPR == 1 && row >= p.rows) return;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (c >= nc) break;
      const int col = col0 + c * WPR * 64 * CH;
      if (col < p.cols) in.x[c].load(xs + row * ldx + col, left(col));
    }
    if (SECOND) {
      in.r = p.r64[row];
    } else if (p.res) {
#pragma unroll
      for (int c = 0; c < N; ++c) {
        if (c >= nc) break;
        const int col = col0 + c * WPR * 64 * CH;
        if (col < p.cols) in.res[c].load(static_cast<const T*>(p.res) + row * p.ldr + col, left(col));
      }
    }
  };
  In next;
  load(next, row_of(blockIdx.x));  // (the first row, on its way meanwhile)
  uint32_t most = 0;
  TensorScale ts = {1.0f, 0.0f, s_rec};
  if constexpr (EMIT == EMIT_NVFP4) {
    if (SECOND) {
      uint32_t m = 0;
      auto maximum = [&](int i) { return __float_as_uint(p.maxima[min(i, p.n_max - 1)]); };
      m = maximum(threadIdx.x);
      if (p.n_max > WAVES * 64) {
#pragma unroll
        for (int i = 1; i < MAX_WGS / (WAVES * 64); ++i) m = max(m, maximum(i * WAVES * 64 + threadIdx.x));
      }
      m = wave_max(m);
      if (lane == 0) s_max[wave] = m;
      __syncthreads();
      m = 0;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) m = max(m, s_max[i]);
      ts.t = nv_tensor_scale(__uint_as_float(m));
      if (blockIdx.x == 0 && threadIdx.x == 0) *p.tscale = ts.t;
    } else {
      ts.t = *p.tscale;
    }
    if (ts.t >= 0x1p-80f && ts.t <= 0x1p80f) {
      ts.rt = 1.0f / ts.t;
      if (threadIdx.x < 128) {
        const float d = e4m3_value(threadIdx.x) * ts.t;
        s_rec[threadIdx.x] = d > 0.0f ? 1.0f / d : 0.0f;
      }
    }
    __syncthreads();
  }
  // What does not change from row to row: the weights of few chunks, and where a
  // chunk's codes and scale stand in row 0 of a block of rows.
  constexpr bool KEEP = N <= 2;
  constexpr int FMT = EMIT == EMIT_NVFP4 ? FP4Q_NVFP4 : FP4Q_MXFP4, BLK = FMT == FP4Q_NVFP4 ? 16 : 32;
  double kept[KEEP ? N : 1][CH];
  int64_t code0[N], scale0[N];
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const int col = col0 + c * WPR * 64 * CH;
    if (c >= nc || col >= p.cols) continue;
    if (KEEP) {
      float w[CH];
      load_any(p.w, col, p.w_f32, EMIT == EMIT_Y ? p.cols - col : CH, w);
#pragma unroll
      for (int i = 0; i < CH; ++i) kept[KEEP ? c : 0][i] = w[i];
    }
    code0[c] = code_off(p.tiled, 0, col >> 1, p.cols);
    scale0[c] = scale_off<FMT>(p.tiled, 0, col / BLK, p.cols);
  }
  // Few chunks: the next row is on its way while one is worked on (second pass of
  // 8192 x 4096 26.2 us, 27.6 without).
  constexpr bool AHEAD = N <= 2;
  int turn = 0;
  for (int64_t gi = blockIdx.x; gi < p.groups; gi += gridDim.x, turn ^= 1) {
    const int64_t row = row_of(gi);
    if (!AHEAD && gi != blockIdx.x) load(next, row);
    In in = next;
    if (AHEAD && gi + gridDim.x < p.groups) load(next, row_of(gi + gridDim.x));
    if (WPR == 1 && row >= p.rows) continue;
    Raw<T>(&h)[N] = in.x;
    double r;
    if (SECOND) {
      r = in.r;
    } else {
      double ss = 0.0;
      if (p.res) {
        T* out = static_cast<T*>(p.h) + row * p.ldh;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if (c >= nc) break;
          const int col = col0 + c * WPR * 64 * CH;
          if (col >= p.cols) continue;
          float f[CH];
#pragma unroll
          for (int i = 0; i < CH; ++i) f[i] = h[c].at(i) + in.res[c].at(i);
          h[c].set(f);
          h[c].store(out + col, left(col));
        }
      }
#pragma unroll
      for (int c = 0; c < N; ++c) {
        if (c >= nc) break;
        if (col0 + c * WPR * 64 * CH >= p.cols) continue;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const double v = h[c].at(i);
          ss = __builtin_fma(v, v, ss);
        }
      }
      ss = wave_sum(ss);
      if (WPR > 1) {
        if (lane == 0) s_sum[turn][wave] = ss;
        __syncthreads();
        ss = 0.0;
#pragma unroll
        for (int i = 0; i < WPR; ++i) ss += s_sum[turn][i];
      }
      r = 1.0 / sqrt(ss / (double)p.cols + p.eps);
      if (lane == 0 && sub == 0) {
        if (EMIT == EMIT_MAX) p.r64[row] = r;
        if (p.rstd) p.rstd[row] = (float)r;
      }
    }
    const int64_t code_row = code_off(p.tiled, row, 0, p.cols), scale_row = scale_off<FMT>(p.tiled, row, 0, p.cols);
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (c >= nc) break;
      const int col = col0 + c * WPR * 64 * CH, n = left(col);
      if (col >= p.cols) continue;
      float w[CH], f[CH];
      if (!KEEP) load_any(p.w, col, p.w_f32, n, w);
#pragma unroll
      for (int i = 0; i < CH; ++i)  // (the first product is exact)
        f[i] = (float)((double)h[c].at(i) * (KEEP ? kept[KEEP ? c : 0][i] : (double)w[i]) * r);
      if (EMIT != EMIT_MAX && p.y) store_any(p.y, row * p.ldy + col, p.y_f32, n, f);
      if constexpr (EMIT != EMIT_Y) {
        Raw<uint16_t> y;
        y.set(f);
        const uint32_t m = max_bits(y);
        if constexpr (EMIT == EMIT_MAX) {
          most = max(most, m);
        } else {
          uint32_t code[2];
          const uint32_t s = encode<EMIT, !SECOND>(y, block_max<EMIT == EMIT_NVFP4 ? 2 : 4>(m), ts, code);
          if constexpr (EMIT == EMIT_MXFP8) {
            *reinterpret_cast<u32x2*>(p.q + row * p.cols + col) = u32x2{code[0], code[1]};
            if ((lane & 3) == 0) p.scales[row * (p.cols / 32) + col / 32] = (uint8_t)s;
          } else {
            *reinterpret_cast<uint32_t*>(p.q + code_row + code0[c]) = code[0];
            if (col % BLK == 0) p.scales[scale_row + scale0[c]] = (uint8_t)s;
            if (p.n_chan > 0) {
              *reinterpret_cast<u32x4*>(ys + col) = y.v;
              codes[col / CH] = code[0];
              scs[col / CH] = (uint8_t)s;
            }
          }
        }
      }
    }
    if (QUANT && EMIT != EMIT_MXFP8 && p.n_chan > 0) {
      if (WPR > 1) __syncthreads();
      else wave_fence();
      for (int j = sub * 64 + lane; j < p.n_chan; j += WPR * 64) {
        const uint32_t ch = min((uint32_t)p.chan[j], (uint32_t)p.cols - 1);
        const uint32_t e = codes[ch / CH] >> (4 * (ch % CH)) & 15u, s = scs[ch / CH];
        const float mag = e2m1_mag_value(e & 7u) * (EMIT == EMIT_NVFP4 ? e4m3_value(s) : exp2i((int)s - 127)) * ts.t;
        const f32x2n d = {bf16_to_f32(ys[ch]) - (e & 8u ? -mag : mag), 0.0f};
        p.resid[row * p.n_chan + j] = (uint16_t)__builtin_bit_cast(uint32_t, __builtin_convertvector(d, bf16x2n));
      }
      if (WPR > 1) __syncthreads();
      else wave_fence();
    }
  }
  if constexpr (EMIT == EMIT_MAX) {
    most = wave_max(most);
    if (lane == 0) s_max[wave] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < WAVES; ++i) most = max(most, s_max[i]);
      p.maxima[blockIdx.x] = bf16_to_f32(most);
    }
  }
}

// ---- the gradient -----------------------------------------------------------
//
// With u = h r and g = weight d_y:  d_x = r (g - u mean(g u)) + d_h,
// d_weight = sum over the rows of d_y u.  Four or eight waves take a row at a time; a
// lane adds up its columns' d_weight over the workgroup's rows, and a second
// kernel adds the workgroups' sums, always in the same order.
struct NormGradArgs {
  const void* h;
  int64_t ldh;
  const void* w;
  int w_f32;
  const float* rstd;
  const void* dy;
  int64_t lddy;
  int dy_f32;
  const void* dh;  // or null
  int64_t lddh;
  void* dx;
  int64_t lddx;
  float* part;     // [gridDim.x][cols]
  int64_t rows;
  int cols;
};

template <typename T, int WPR, int N>
__global__ __launch_bounds__(64 * WPR) void k_norm_backward(NormGradArgs p) {
  __shared__ float s_sum[2][WPR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col0 = (wave * 64 + lane) * CH;
  const int nc = (p.cols + WPR * 64 * CH - 1) / (WPR * 64 * CH);
  float dw[N][CH];
#pragma unroll
  for (int c = 0; c < N; ++c)
#pragma unroll
    for (int i = 0; i < CH; ++i) dw[c][i] = 0.0f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const float r = p.rstd[row];
    Raw<T> hr[N], dh[N];
    float g[N][CH];
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (c >= nc) break;
      const int col = col0 + c * WPR * 64 * CH, n = p.cols - col;
      if (n <= 0) continue;
      hr[c].load(static_cast<const T*>(p.h) + row * p.ldh + col, n);
      load_any(p.dy, row * p.lddy + col, p.dy_f32, n, g[c]);
      if (p.dh) dh[c].load(static_cast<const T*>(p.dh) + row * p.lddh + col, n);
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (c >= nc) break;
      const int col = col0 + c * WPR * 64 * CH, n = p.cols - col;
      if (n <= 0) continue;
      float w[CH];
      load_any(p.w, col, p.w_f32, n, w);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const float u = hr[c].at(i) * r;
        dw[c][i] = __builtin_fmaf(g[c][i], u, dw[c][i]);
        g[c][i] *= w[i];
        sum = __builtin_fmaf(g[c][i], u, sum);
      }
    }
    sum = wave_sum(sum);
    if (lane == 0) s_sum[turn][wave] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) sum += s_sum[turn][i];
    sum /= (float)p.cols;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (c >= nc) break;
      const int col = col0 + c * WPR * 64 * CH, n = p.cols - col;
      if (n <= 0) continue;
      float f[CH];
#pragma unroll
      for (int i = 0; i < CH; ++i) f[i] = r * __builtin_fmaf(-(hr[c].at(i) * r), sum, g[c][i]);
      if (p.dh) {
#pragma unroll
        for (int i = 0; i < CH; ++i) f[i] += dh[c].at(i);
      }
      Raw<T> o;
      o.set(f);
      o.store(dx + col, n);
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    if (c >= nc) break;
    const int col = col0 + c * WPR * 64 * CH, n = p.cols - col;
    if (n <= 0) continue;
    Raw<float> o;
    o.set(dw[c]);
    o.store(part + col, n);
  }
}

// d_weight from the workgroups' sums: 16 columns a workgroup, 16 threads on each.
__global__ __launch_bounds__(256) void k_norm_dweight(const float* __restrict__ part, int n, int cols,
                                                      float* __restrict__ dw) {
  __shared__ float s[16][16];
  const int c = threadIdx.x & 15, k = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float sum = 0.0f;
  if (col < cols) {
#pragma unroll 8
    for (int i = k; i < n; i += 16) sum += part[(int64_t)i * cols + col];
  }
  s[k][c] = sum;
  __syncthreads();
  if (k > 0 || col >= cols) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) sum += s[i][c];
  dw[col] = sum;
}

// ---- the values of an operand -------------------------------------------------
//
// A lane takes eight codes; a workgroup 16 rows of 512 columns, so that a tiled
// block's lines are read by one.
template <int EMIT>
__global__ __launch_bounds__(256) void k_dequantize(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales,
                                                    const float* __restrict__ tscale, bool tiled, int64_t rows,
                                                    int64_t cols, void* __restrict__ y, int y_f32, int64_t ldy,
                                                    uint32_t col_blocks) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)(blockIdx.x % col_blocks) * 512 + lane * CH;
  const int64_t row0 = (int64_t)(blockIdx.x / col_blocks) * 16 + wave * 4;
  if (col >= cols) return;
  const float t = EMIT == EMIT_NVFP4 ? *tscale : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + i;
    if (row >= rows) break;
    float f[CH];
    if constexpr (EMIT == EMIT_MXFP8) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(q + row * cols + col);
      const float s = exp2i((int)scales[row * (cols / 32) + col / 32] - 127);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f32x2n a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k], false);
        const f32x2n b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k], true);
        f[4 * k] = a[0] * s;
        f[4 * k + 1] = a[1] * s;
        f[4 * k + 2] = b[0] * s;
        f[4 * k + 3] = b[1] * s;
      }
    } else {
      constexpr int FMT = EMIT == EMIT_NVFP4 ? FP4Q_NVFP4 : FP4Q_MXFP4, BLK = FMT == FP4Q_NVFP4 ? 16 : 32;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(q + code_off(tiled, row, col >> 1, cols));
      const uint32_t sc = scales[scale_off<FMT>(tiled, row, col / BLK, cols)];
      const float s = EMIT == EMIT_NVFP4 ? e4m3_value(sc) : exp2i((int)sc - 127);
#define FP4Q_PAIR(N)                                                                  \
  {                                                                                   \
    const f32x2n e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, N);            \
    f[2 * N] = (e[0] * s) * t;                                                        \
    f[2 * N + 1] = (e[1] * s) * t;                                                    \
  }
      FP4Q_PAIR(0) FP4Q_PAIR(1) FP4Q_PAIR(2) FP4Q_PAIR(3)
#undef FP4Q_PAIR
    }
    store_any(y, row * ldy + col, y_f32, CH, f);
  }
}

// The tensor scale of no rows.
__global__ void k_scale_one(float* tscale) { *tscale = 1.0f; }

template <typename T, int WPR, int N, int EMIT, bool SECOND>
int launch_pass(NormArgs p, hipStream_t stream) {
  constexpr int ROWS = WPR == 1 ? 4 : 1;
  p.groups = (p.rows + ROWS - 1) / ROWS;
  const int grid = (int)(p.groups < MAX_WGS ? p.groups : MAX_WGS);
  const size_t lds = EMIT >= EMIT_NVFP4 && p.n_chan > 0 ? (size_t)ROWS * p.cols * 4 : 0;
  hipLaunchKernelGGL((k_norm<T, WPR, N, EMIT, SECOND>), dim3(grid), dim3(WPR == 8 ? 512 : 256), lds, stream, p);
  return grid;
}

template <typename T, int WPR, int N>
void launch_emit(NormArgs p, int emit, bool given, hipStream_t stream) {
  if (emit == EMIT_Y) {
    launch_pass<T, WPR, N, EMIT_Y, false>(p, stream);
  } else if (emit == EMIT_MXFP4) {
    launch_pass<T, WPR, N, EMIT_MXFP4, false>(p, stream);
  } else if (emit == EMIT_MXFP8) {
    launch_pass<T, WPR, N, EMIT_MXFP8, false>(p, stream);
  } else if (given) {
    launch_pass<T, WPR, N, EMIT_NVFP4, false>(p, stream);
  } else {
    p.n_max = launch_pass<T, WPR, N, EMIT_MAX, false>(p, stream);
    p.rstd = nullptr;
    launch_pass<T, WPR, N, EMIT_NVFP4, true>(p, stream);
  }
}

// Waves of a row and chunks of a lane.  A wave, and no barrier, for rows of up to 1024
// columns from 1024 rows on: 16384 x 1024 36 us (NVFP4), by four waves 54; 1024 x 1024
// 8.4 and 8.7, x 512 7.1 and 8.4; 512 x 1024 8.2 and 8.0, 64 x 1024 8.0 and 7.3.  Longer
// rows in a wave take its registers: 8192 x 4096 (MXFP8) 54, by four waves 43.
template <typename T>
void launch_type(const NormArgs& p, int emit, bool given, hipStream_t stream) {
  if (p.rows >= 1024 && p.cols <= room(1, 2)) launch_emit<T, 1, 2>(p, emit, given, stream);
  else if (p.cols <= room(4, 2)) launch_emit<T, 4, 2>(p, emit, given, stream);
  else if (p.cols <= room(4, 4)) launch_emit<T, 4, 4>(p, emit, given, stream);
  else if (p.cols <= room(8, 4)) launch_emit<T, 8, 4>(p, emit, given, stream);
  else launch_emit<T, 8, 8>(p, emit, given, stream);
}

// Workgroups, each with a row of d_weight's sums: four rows each, between 256 and 1024 of
// them.  us for that, for 512 and for 1024 at least: 512 x 4096 13.4, 16.2, 16.2; 1024 x
// 4096 16.6, 16.0, 20.1; 700 x 1024 8.0, 8.7, 10.0.  At most 512: 8192 x 4096 71, for 61.
int backward_blocks(int64_t rows) {
  const int64_t n = rows / 4 < 256 ? 256 : rows / 4 < 1024 ? rows / 4 : 1024;
  return (int)(rows < n ? rows : n);
}

template <typename T>
void launch_backward_type(const NormGradArgs& p, hipStream_t stream) {
  const dim3 grid(backward_blocks(p.rows));
  if (p.cols <= room(4, 2)) hipLaunchKernelGGL((k_norm_backward<T, 4, 2>), grid, dim3(256), 0, stream, p);
  else if (p.cols <= room(4, 4)) hipLaunchKernelGGL((k_norm_backward<T, 4, 4>), grid, dim3(256), 0, stream, p);
  else if (p.cols <= room(8, 4)) hipLaunchKernelGGL((k_norm_backward<T, 8, 4>), grid, dim3(512), 0, stream, p);
  else hipLaunchKernelGGL((k_norm_backward<T, 8, 8>), grid, dim3(512), 0, stream, p);
}

}  // namespace

int norm_max_cols() { return room(8, 8); }

// First of the second pass's inputs: the rows' r; then the maxima.
size_t norm_workspace_bytes(int64_t rows) { return (size_t)rows * 8 + MAX_WGS * 4; }

void launch_norm(int f32, const void* x, int64_t ldx, const void* res, int64_t ldr, void* h, int64_t ldh,
                 const void* w, int w_f32, double eps, int64_t rows, int cols, void* y, int y_f32, int64_t ldy,
                 float* rstd, int fmt, bool tiled, uint8_t* q, uint8_t* scales, float* tscale, bool given,
                 const int32_t* chan, int n_chan, uint16_t* resid, void* ws, hipStream_t stream) {
  NormArgs p = {};
  p.x = x;
  p.ldx = ldx;
  p.res = res;
  p.ldr = ldr;
  p.h = h;
  p.ldh = ldh;
  p.w = w;
  p.w_f32 = w_f32;
  p.eps = eps;
  p.rows = rows;
  p.cols = cols;
  p.y = y;
  p.ldy = ldy;
  p.y_f32 = y_f32;
  p.rstd = rstd;
  p.q = q;
  p.scales = scales;
  p.tscale = tscale;
  p.tiled = tiled;
  p.chan = chan;
  p.n_chan = n_chan;
  p.resid = resid;
  p.r64 = static_cast<double*>(ws);
  p.maxima = reinterpret_cast<float*>(p.r64 + rows);
  if (rows == 0) {
    if (fmt == FP4Q_NVFP4 && !given) hipLaunchKernelGGL(k_scale_one, dim3(1), dim3(1), 0, stream, tscale);
    return;
  }
  const int emit = fmt < 0 ? EMIT_Y : fmt == FP4Q_NVFP4 ? EMIT_NVFP4 : fmt == FP4Q_MXFP4 ? EMIT_MXFP4 : EMIT_MXFP8;
  if (f32) launch_type<float>(p, emit, given, stream);
  else launch_type<uint16_t>(p, emit, given, stream);
}

size_t norm_backward_workspace_bytes(int64_t rows, int cols) {
  return (size_t)backward_blocks(rows) * (size_t)cols * 4;
}

void launch_norm_backward(int f32, const void* h, int64_t ldh, const void* w, int w_f32, const float* rstd,
                          const void* dy, int dy_f32, int64_t lddy, const void* dh, int64_t lddh, void* dx,
                          int64_t lddx, float* dw, int64_t rows, int cols, void* ws, hipStream_t stream) {
  const NormGradArgs p = {h, ldh, w, w_f32, rstd, dy, lddy, dy_f32, dh, lddh, dx, lddx, static_cast<float*>(ws),
                          rows, cols};
  const int n = backward_blocks(rows);
  if (n > 0) {
    if (f32) launch_backward_type<float>(p, stream);
    else launch_backward_type<uint16_t>(p, stream);
  }
  hipLaunchKernelGGL(k_norm_dweight, dim3((cols + 15) / 16), dim3(256), 0, stream, p.part, n, cols, dw);
}

void launch_dequantize(int fmt, bool tiled, const uint8_t* q, const uint8_t* scales, const float* tscale,
                       int64_t rows, int64_t cols, void* y, int y_f32, int64_t ldy, hipStream_t stream) {
  const uint32_t cb = (uint32_t)((cols + 511) / 512);
  const dim3 grid((unsigned)((rows + 15) / 16 * cb));
  if (fmt == FP4Q_NVFP4)
    hipLaunchKernelGGL(k_dequantize<EMIT_NVFP4>, grid, dim3(256), 0, stream, q, scales, tscale, tiled, rows, cols,
                       y, y_f32, ldy, cb);
  else if (fmt == FP4Q_MXFP4)
    hipLaunchKernelGGL(k_dequantize<EMIT_MXFP4>, grid, dim3(256), 0, stream, q, scales, tscale, tiled, rows, cols,
                       y, y_f32, ldy, cb);
  else
    hipLaunchKernelGGL(k_dequantize<EMIT_MXFP8>, grid, dim3(256), 0, stream, q, scales, tscale, tiled, rows, cols,
                       y, y_f32, ldy, cb);
}

}  // namespace fp4q
