// kvcache.hip -- the paged FP4 key/value cache: quantize new tokens into it
// and read them back (layout and rules in include/fp4q.h).
//
// Both kernels give a thread 32 consecutive elements of one (token, head):
// two NVFP4 blocks or one MXFP4 block.  In a V row the byte of elements
// (32j + l, 32j + 16 + l) stands at (l * 4 + token % 4) * D/32 + j of its
// four-token group, so the 16 bytes of a thread's run interleave with those
// of the other runs and of the three neighbouring tokens.  Every byte belongs
// to one token: an append touches no other token's bytes.
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

// The 16 bytes of a V run are byte-interleaved; w holds the codes of the run
// two neighbouring elements to a byte, b the bytes of elements (l, 16 + l).
__device__ __forceinline__ void v_bytes_from_codes(const uint32_t (&w)[4], uint8_t (&b)[16]) {
#pragma unroll
  for (int l = 0; l < 16; ++l) {
    const uint32_t lo = (w[l >> 3] >> (4 * (l & 7))) & 15u;
    const uint32_t hi = (w[2 + (l >> 3)] >> (4 * (l & 7))) & 15u;
    b[l] = (uint8_t)(lo | (hi << 4));
  }
}

__device__ __forceinline__ void v_codes_from_bytes(const uint8_t (&b)[16], uint32_t (&w)[4]) {
  w[0] = w[1] = w[2] = w[3] = 0;
#pragma unroll
  for (int l = 0; l < 16; ++l) {
    w[l >> 3] |= (uint32_t)(b[l] & 15u) << (4 * (l & 7));
    w[2 + (l >> 3)] |= (uint32_t)(b[l] >> 4) << (4 * (l & 7));
  }
}

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
      s |= sb << (8 * blk);
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
  const KvItem it = kv_item<FMT, D>(p, s_off);
  if (it.base == nullptr) return;
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
    uint8_t b[16];
    v_bytes_from_codes(w, b);
    uint8_t* dst = it.base + L::v_codes(page) + (it.slot >> 2) * (2 * D) + (it.slot & 3) * L::J + it.j;
#pragma unroll
    for (int l = 0; l < 16; ++l) dst[l * 4 * L::J] = b[l];
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(KV_THREADS) void k_kv_read(KvArgs p) {
  typedef KvLayout<FMT, D> L;
  __shared__ int32_t s_off[KV_LDS_SEQ + 1];
  const KvItem it = kv_item<FMT, D>(p, s_off);
  if (it.row >= p.rows) return;
  const bool is_v = blockIdx.y != 0;
  uint16_t* dst = is_v ? p.v + it.row * p.ldv : p.k + it.row * p.ldk;
  u32x4* y4 = reinterpret_cast<u32x4*>(dst + it.h * D + it.j * 32);
  if (it.base == nullptr) {  // nothing stored for this row
    const u32x4 z = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) y4[i] = z;
    return;
  }
  const int page = 1 << p.page_shift;
  uint32_t w[4];
  if (!is_v) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(it.base + it.slot * (D / 2) + it.j * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = u[i];
  } else {
    uint8_t b[16];
    const uint8_t* src =
        it.base + L::v_codes(page) + (it.slot >> 2) * (2 * D) + (it.slot & 3) * L::J + it.j;
#pragma unroll
    for (int l = 0; l < 16; ++l) b[l] = src[l * 4 * L::J];
    v_codes_from_bytes(b, w);
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
    u32x4 o;
#define FP4Q_KV_PAIR(N)                                                             \
  {                                                                                 \
    const v2f32k e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, N);       \
    v2f32k f;                                                                       \
    f[0] = (e[0] * s) * t;                                                          \
    f[1] = (e[1] * s) * t;                                                          \
    o[N] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2k));       \
  }
    FP4Q_KV_PAIR(0) FP4Q_KV_PAIR(1) FP4Q_KV_PAIR(2) FP4Q_KV_PAIR(3)
#undef FP4Q_KV_PAIR
    y4[i] = o;
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
