// kvcache.hip -- the paged FP4 key/value cache: quantize new tokens into it
// and read them back (layout and rules in include/fp4q.h).
//
// Both kernels give a thread 32 consecutive elements of one (token, head):
// two NVFP4 blocks or one MXFP4 block.  In a V row the byte of elements
// (32j + l, 32j + 16 + l) stands at (l * 4 + token % 4) * D/32 + j of its
// four-token group, so the 16 bytes of a thread's run interleave with those
// of the other runs and of the three neighbouring tokens.  Every byte belongs
// to one token: an append touches no other token's bytes.  Both are bound by
// HBM: 12.4 thousand tokens (8 heads of 128, MXFP4: 64 MB each way) take 14 us
// each, 4.6 TB/s; 64 tokens 5.3 and 4.2 us, the chain of a search, a table entry
// and a line.
#include "fp4q_device.h"
#include "fp4q_internal.h"
#include "kv_layout.h"

namespace fp4q {

namespace {

constexpr int KV_THREADS = 256;
constexpr int KV_LDS_SEQ = 2048;  // offsets kept in LDS up to this many sequences

typedef __bf16 bf16x2k __attribute__((ext_vector_type(2)));
typedef float v2f32k __attribute__((ext_vector_type(2)));

struct KvArgs {
  uint8_t* cache;
  int64_t n_pages;
  int page_shift, H;
  const int32_t* off;
  int B;
  const int32_t* table;
  int64_t ldt, table_cols;
  const int32_t* lens;
  int64_t rows;
  uint16_t* k;
  uint16_t* v;
  int64_t ldk, ldv;
  const float* kts;
  const float* vts;
};

// This thread's (row, head, run), its cache bytes (null: no such row, or its
// page is not in the cache) and the token's place in the page.
struct KvItem {
  int64_t row;
  int h, j, slot;
  uint8_t* base;
};

template <int FMT, int D>
__device__ __forceinline__ KvItem kv_item(const KvArgs& p, int32_t* s_off) {
  typedef KvLayout<FMT, D> L;
  const int32_t* off = p.off;
  if (p.B <= KV_LDS_SEQ) {  // search in LDS: a step costs an LDS read, not an L2 one
    for (int i = threadIdx.x; i <= p.B; i += KV_THREADS) s_off[i] = p.off[i];
    __syncthreads();
    off = s_off;
  }
  // runs fastest, then four neighbouring rows, then heads: the four tokens of
  // a V group are written by one wave
  const uint32_t idx = blockIdx.x * KV_THREADS + threadIdx.x;
  KvItem it;
  it.j = (int)(idx % L::J);
  const uint32_t a = idx / L::J, c = a >> 2;
  it.h = (int)(c % (uint32_t)p.H);
  it.row = (int64_t)(c / (uint32_t)p.H) * 4 + (a & 3);
  it.base = nullptr;
  it.slot = 0;
  if (it.row < p.rows && it.row >= off[0] && it.row < off[p.B]) {
    const int b = kv_sequence(off, p.B, it.row);
    const int64_t pos = (int64_t)p.lens[b] - off[b + 1] + it.row;
    const int64_t pg = pos >> p.page_shift;
    if (pos >= 0 && pg < p.table_cols) {
      const int64_t id = p.table[b * p.ldt + pg];
      if (id >= 0 && id < p.n_pages) {
        const int page = 1 << p.page_shift;
        it.slot = (int)(pos & (page - 1));
        it.base = p.cache + (id * p.H + it.h) * (int64_t)L::bytes(page);
      }
    }
  }
  return it;
}

// A V run is stored with its bytes apart: byte l (elements l, 16 + l of the run)
// of run j of a token at l * 4J + j, so the J lanes that hold a token's runs
// exchange bytes through LDS, after which a lane has 16 / J stretches of J bytes
// that lie together in the cache.  w: the run's codes, two neighbouring elements
// to a byte; b: bytes (16 / J) j .. of the token, each J long.
template <int J>
__device__ __forceinline__ u32x4 v_bytes_from_codes(const uint32_t (&w)[4], int j, uint8_t* token) {
#pragma unroll
  for (int l = 0; l < 16; ++l) {
    const uint32_t lo = (w[l >> 3] >> (4 * (l & 7))) & 15u;
    const uint32_t hi = (w[2 + (l >> 3)] >> (4 * (l & 7))) & 15u;
    token[l * J + j] = (uint8_t)(lo | (hi << 4));
  }
  wave_fence();
  return *reinterpret_cast<const u32x4*>(token + 16 * j);
}

template <int J>
__device__ __forceinline__ void v_codes_from_bytes(u32x4 b, int j, uint8_t* token, uint32_t (&w)[4]) {
  *reinterpret_cast<u32x4*>(token + 16 * j) = b;
  wave_fence();
  w[0] = w[1] = w[2] = w[3] = 0;
#pragma unroll
  for (int l = 0; l < 16; ++l) {
    const uint32_t c = token[l * J + j];
    w[l >> 3] |= (c & 15u) << (4 * (l & 7));
    w[2 + (l >> 3)] |= (c >> 4) << (4 * (l & 7));
  }
}

// The stretches of lane j: J bytes each, 4J apart in the cache.
template <int J>
struct Stretch;
template <> struct Stretch<2> { typedef uint16_t type; };
template <> struct Stretch<4> { typedef uint32_t type; };
template <> struct Stretch<8> { typedef u32x2 type; };

// Codes (w) and scale codes (s: NVFP4 two bytes, MXFP4 one) of 32 elements.
template <int FMT>
__device__ __forceinline__ void quant32(const uint32_t (&x)[16], float t, uint32_t (&w)[4],
                                        uint32_t& s) {
  constexpr int NB = FMT == FP4Q_NVFP4 ? 2 : 1;
  s = 0;
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    uint32_t m = 0;  // the largest magnitude, as BF16 bits
#pragma unroll
    for (int i = 0; i < 16 / NB; ++i) {
      const uint32_t u = x[blk * 8 + i];
      m = max(m, max(u & 0x7FFFu, (u >> 16) & 0x7FFFu));
    }
    const float amax = bf16_to_f32(m);
    float v[8];
    if (FMT == FP4Q_NVFP4) {
      const uint32_t sb = e4m3_encode((amax / 6.0f) / t);
      s |= (sb & 0xFFu) << (8 * blk);  // (more than a byte for a NaN, which must not reach the other block)
      const float d = e4m3_value(sb) * t;
      // quot_rn's range; its operands are held within 8 d (beyond it every
      // quotient gives the largest code)
      const bool fast = d >= 0x1p-96f && d <= 0x1p96f;
      const float y = fast ? 1.0f / d : 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t u = x[blk * 8 + c * 4 + i / 2];
          const float e = bf16_to_f32((i & 1) ? (u >> 16) : (u & 0xFFFFu));
          if (fast) v[i] = quot_rn(fminf(fmaxf(e, -8.0f * d), 8.0f * d), d, y);
          else v[i] = d > 0.0f ? e / d : 0.0f * e;
        }
        w[blk * 2 + c] = e2m1_pack8(v);
      }
    } else {
      const int e8 = mx_exponent(amax);
      s = (uint32_t)(e8 + 127);
      const float sc = __uint_as_float(s << 23);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t u = x[c * 4 + i / 2];
          v[i] = bf16_to_f32((i & 1) ? (u >> 16) : (u & 0xFFFFu));
        }
        w[c] = e2m1_pack8(v, sc);
      }
    }
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(KV_THREADS) void k_kv_append(KvArgs p) {
  typedef KvLayout<FMT, D> L;
  __shared__ int32_t s_off[KV_LDS_SEQ + 1];
  __shared__ __attribute__((aligned(16))) uint8_t s_v[KV_THREADS * 16];
  const KvItem it = kv_item<FMT, D>(p, s_off);
  if (it.base == nullptr) return;  // (the lanes of a token together)
  const bool is_v = blockIdx.y != 0;
  const uint16_t* src = is_v ? p.v + it.row * p.ldv : p.k + it.row * p.ldk;
  const u32x4* x4 = reinterpret_cast<const u32x4*>(src + it.h * D + it.j * 32);
  uint32_t x[16], w[4], s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x4 u = x4[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * i + e] = u[e];
  }
  const float t = FMT == FP4Q_NVFP4 ? (is_v ? p.vts : p.kts)[it.h] : 1.0f;
  quant32<FMT>(x, t, w, s);
  const int page = 1 << p.page_shift;
  uint8_t* sc = it.base + (is_v ? L::v_scales(page) : L::k_scales(page)) + it.slot * L::SB;
  if (FMT == FP4Q_NVFP4) reinterpret_cast<uint16_t*>(sc)[it.j] = (uint16_t)s;
  else sc[it.j] = (uint8_t)s;
  if (!is_v) {
    u32x4 o = {w[0], w[1], w[2], w[3]};
    *reinterpret_cast<u32x4*>(it.base + it.slot * (D / 2) + it.j * 16) = o;
  } else {
    typedef typename Stretch<L::J>::type T;
    const u32x4 b = v_bytes_from_codes<L::J>(w, it.j, s_v + threadIdx.x / L::J * (16 * L::J));
    uint8_t* dst = it.base + L::v_codes(page) + (it.slot >> 2) * (2 * D) + (it.slot & 3) * L::J +
                   it.j * (16 / L::J) * 4 * L::J;
#pragma unroll
    for (int i = 0; i < 16 / L::J; ++i) {
      T t;
      if constexpr (L::J == 2) t = (T)(b[i >> 1] >> (16 * (i & 1)));
      else if constexpr (L::J == 4) t = b[i];
      else t = T{b[2 * i], b[2 * i + 1]};
      *reinterpret_cast<T*>(dst + i * 4 * L::J) = t;
    }
  }
}

// A thread's 64 bytes leave through LDS, so that four lanes write each of them
// at once (stored from the registers that hold them they took half as long again).
template <int FMT, int D>
__global__ __launch_bounds__(KV_THREADS) void k_kv_read(KvArgs p) {
  typedef KvLayout<FMT, D> L;
  __shared__ int32_t s_off[KV_LDS_SEQ + 1];
  __shared__ u32x4 s_out[KV_THREADS * 4];
  __shared__ u32x4* s_dst[KV_THREADS];
  uint8_t* const s_v = reinterpret_cast<uint8_t*>(s_out + (threadIdx.x & ~63) * 4);  // the wave's part
  const KvItem it = kv_item<FMT, D>(p, s_off);
  const bool is_v = blockIdx.y != 0;
  const int lane = threadIdx.x & 63;
  {
    uint16_t* dst = is_v ? p.v + it.row * p.ldv : p.k + it.row * p.ldk;
    s_dst[threadIdx.x] = it.row < p.rows ? reinterpret_cast<u32x4*>(dst + it.h * D + it.j * 32) : nullptr;
  }
  u32x4 out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = u32x4{0, 0, 0, 0};  // nothing stored for this row: zeros
  if (it.base != nullptr) {
    const int page = 1 << p.page_shift;
    uint32_t w[4];
    if (!is_v) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(it.base + it.slot * (D / 2) + it.j * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = u[i];
    } else {
      typedef typename Stretch<L::J>::type T;
      const uint8_t* src = it.base + L::v_codes(page) + (it.slot >> 2) * (2 * D) + (it.slot & 3) * L::J +
                           it.j * (16 / L::J) * 4 * L::J;
      u32x4 b = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16 / L::J; ++i) {
        const T t = *reinterpret_cast<const T*>(src + i * 4 * L::J);
        if constexpr (L::J == 2) {
          b[i >> 1] |= (uint32_t)t << (16 * (i & 1));
        } else if constexpr (L::J == 4) {
          b[i] = t;
        } else {
          b[2 * i] = t[0];
          b[2 * i + 1] = t[1];
        }
      }
      v_codes_from_bytes<L::J>(b, it.j, s_v + lane / L::J * (16 * L::J), w);
    }
    const uint8_t* sc = it.base + (is_v ? L::v_scales(page) : L::k_scales(page)) + it.slot * L::SB;
    float s0, s1, t = 1.0f;
    if (FMT == FP4Q_NVFP4) {
      const uint32_t s = reinterpret_cast<const uint16_t*>(sc)[it.j];
      s0 = e4m3_value(s & 0xFFu);
      s1 = e4m3_value(s >> 8);
      t = (is_v ? p.vts : p.kts)[it.h];
    } else {
      s0 = s1 = exp2i((int)sc[it.j] - 127);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = i < 2 ? s0 : s1;
#define FP4Q_KV_PAIR(N)                                                             \
    {                                                                                 \
      const v2f32k e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, N);       \
      v2f32k f;                                                                       \
      f[0] = (e[0] * s) * t;                                                          \
      f[1] = (e[1] * s) * t;                                                          \
      out[i][N] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2k));       \
    }
      FP4Q_KV_PAIR(0) FP4Q_KV_PAIR(1) FP4Q_KV_PAIR(2) FP4Q_KV_PAIR(3)
#undef FP4Q_KV_PAIR
    }
  }
  wave_fence();
  // chunk i of a lane's four, turned by its number so that the banks are all used
  u32x4* const mine = s_out + (threadIdx.x & ~63) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) mine[lane * 4 + ((i + (lane >> 2)) & 3)] = out[i];
  wave_fence();
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int from = 16 * m + (lane >> 2), i = lane & 3;
    u32x4* dst = s_dst[(threadIdx.x & ~63) + from];
    if (dst) dst[i] = mine[from * 4 + ((i + (from >> 2)) & 3)];
  }
}

template <int FMT, int D>
void launch(bool append, const KvArgs& p, hipStream_t stream) {
  const int64_t items = (p.rows + 3) / 4 * 4 * p.H * (D / 32);
  const dim3 grid((unsigned)((items + KV_THREADS - 1) / KV_THREADS), 2);
  if (append) hipLaunchKernelGGL((k_kv_append<FMT, D>), grid, dim3(KV_THREADS), 0, stream, p);
  else hipLaunchKernelGGL((k_kv_read<FMT, D>), grid, dim3(KV_THREADS), 0, stream, p);
}

}  // namespace

void launch_kv_copy(bool append, int fmt, uint8_t* cache, int64_t n_pages, int page_shift, int H,
                    int D, const int32_t* off, int B, const int32_t* table, int64_t ldt, int64_t table_cols,
                    const int32_t* lens, int64_t rows, uint16_t* k, int64_t ldk, uint16_t* v,
                    int64_t ldv, const float* kts, const float* vts, hipStream_t stream) {
  const KvArgs p = {cache, n_pages, page_shift, H, off, B, table, ldt, table_cols, lens, rows,
                    k,     v,       ldk,        ldv, kts, vts};
  if (fmt == FP4Q_NVFP4) {
    if (D == 64) launch<FP4Q_NVFP4, 64>(append, p, stream);
    else if (D == 128) launch<FP4Q_NVFP4, 128>(append, p, stream);
    else launch<FP4Q_NVFP4, 256>(append, p, stream);
  } else {
    if (D == 64) launch<FP4Q_MXFP4, 64>(append, p, stream);
    else if (D == 128) launch<FP4Q_MXFP4, 128>(append, p, stream);
    else launch<FP4Q_MXFP4, 256>(append, p, stream);
  }
}

}  // namespace fp4q
