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
//
// The rotated append turns pairs by position * frequency on the way: a wave a token
// computes its sines once, 64-bit, into LDS and takes all of its heads past them,
// query heads to their output, key heads through LDS into the quantizer.  HBM again:
// 16.3 thousand tokens, half of each head, MXFP4 (369 MB) 81 us, 4.6 TB/s; 64 tokens of
// 32 + 8 heads 6.5 us, the same chain and the sines.
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

// Run j of a token's scale codes, K codes and (as v_bytes_from_codes gives them) V
// bytes into its head's page.
template <int FMT, int D>
__device__ __forceinline__ void store_scales(uint8_t* base, bool is_v, int page, int slot, int j, uint32_t s) {
  typedef KvLayout<FMT, D> L;
  uint8_t* sc = base + (is_v ? L::v_scales(page) : L::k_scales(page)) + slot * L::SB;
  if (FMT == FP4Q_NVFP4) reinterpret_cast<uint16_t*>(sc)[j] = (uint16_t)s;
  else sc[j] = (uint8_t)s;
}

template <int FMT, int D>
__device__ __forceinline__ void store_k(uint8_t* base, int slot, int j, const uint32_t (&w)[4]) {
  const u32x4 o = {w[0], w[1], w[2], w[3]};
  *reinterpret_cast<u32x4*>(base + slot * (D / 2) + j * 16) = o;
}

template <int FMT, int D>
__device__ __forceinline__ void store_v(uint8_t* base, int page, int slot, int j, u32x4 b) {
  typedef KvLayout<FMT, D> L;
  typedef typename Stretch<L::J>::type T;
  uint8_t* dst = base + L::v_codes(page) + (slot >> 2) * (2 * D) + (slot & 3) * L::J + j * (16 / L::J) * 4 * L::J;
#pragma unroll
  for (int i = 0; i < 16 / L::J; ++i) {
    T t;
    if constexpr (L::J == 2) t = (T)(b[i >> 1] >> (16 * (i & 1)));
    else if constexpr (L::J == 4) t = b[i];
    else t = T{b[2 * i], b[2 * i + 1]};
    *reinterpret_cast<T*>(dst + i * 4 * L::J) = t;
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
  store_scales<FMT, D>(it.base, is_v, page, it.slot, it.j, s);
  if (!is_v) {
    store_k<FMT, D>(it.base, it.slot, it.j, w);
  } else {
    const u32x4 b = v_bytes_from_codes<L::J>(w, it.j, s_v + threadIdx.x / L::J * (16 * L::J));
    store_v<FMT, D>(it.base, page, it.slot, it.j, b);
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

// ---- append with the position rotation ----------------------------------------
//
// Queries and keys turn by their positions on the way: with a = position x
// frequency, a pair (x1, x2) becomes (x1 cos a - x2 sin a, x2 cos a + x1 sin a),
// rounded to F32 and then to BF16; keys and values go into the cache by
// quant32's rule.  Angles, their sines and the products are 64-bit: at position
// 10^5 a 32-bit angle is off by 2^-7, and a key next to one of the format's
// borders would take another code than the definition's.
//
// A wave takes a token: its frequencies' sines and cosines are computed once,
// into LDS, for all heads.  A lane then has 16 elements of a head (eight pairs,
// or two chunks of eight that pass) of every 64 / (D/16)-th head, so that its
// sines stay in registers and a wave's loads lie together.  The keys of those
// heads pass through LDS to the lanes that quantize 32 of them.

struct RotArgs {
  KvArgs kv;
  const uint16_t* q;
  uint16_t* qo;
  int64_t ldq, ldqo;
  int heads, half;  // half: pairs of a head that turn (a multiple of 8)
  bool halves;      // pair p: elements p and p + half; else 2p and 2p + 1
  const float* freqs;
  const int32_t* positions;  // or null: by the sequences
  int per;                   // query heads of a part; 0: one part does all
};

// Sine and cosine for |a| < 2^40: a less the nearest multiple of pi/2 (whose
// product with the first 53 bits of pi/2 leaves a exactly), then the Taylor
// series to x^15 and x^16, whose next terms are below 2^-54 on [-pi/4, pi/4].
__device__ __forceinline__ double2 cos_sin(double a) {
  const double n = rint(a * 0.636619772367581343);
  double x = __builtin_fma(-n, 0x1.921fb54442d18p+0, a);
  x = __builtin_fma(-n, 0x1.1a62633145c07p-54, x);
  const double z = x * x;
  double s = -1.0 / 1307674368000.0, c = 1.0 / 20922789888000.0;
  s = __builtin_fma(s, z, 1.0 / 6227020800.0);
  c = __builtin_fma(c, z, -1.0 / 87178291200.0);
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  c = __builtin_fma(c, z, 1.0 / 479001600.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  s = __builtin_fma(s * z, x, x);
  c = __builtin_fma(c, z, -0.5);
  c = __builtin_fma(c, z, 1.0);
  const int k = (int)((int64_t)n & 3);
  const double cc = k & 1 ? s : c, ss = k & 1 ? c : s;
  return make_double2(k == 1 || k == 2 ? -cc : cc, k >= 2 ? -ss : ss);
}

// The sequence of row r by the whole wave, 64 offsets a step; the last step's lanes
// load what the caller needs of a sequence beside them.
struct WaveSequence {
  int b, end, len;  // the sequence, its last row + 1, its length
};

__device__ __forceinline__ WaveSequence wave_sequence(const KvArgs& p, int64_t r, int lane) {
  int lo = 0, n = p.B;
  while (n > 64) {
    const int step = (n + 63) >> 6;
    const int64_t at = (int64_t)lane * step;
    const uint64_t m = __ballot(at < n && p.off[lo + (at < n ? (int)at : 0)] <= r);
    const int k = max(__popcll(m), 1) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  }
  const int mine = lo + min(lane, n - 1);
  const int first = p.off[mine], end = p.off[mine + 1], len = p.lens[mine];
  const int k = max(__popcll(__ballot(lane < n && first <= r)), 1) - 1;
  return {lo + k, __builtin_amdgcn_readlane(end, k), __builtin_amdgcn_readlane(len, k)};
}

// Eight pairs: chunk a with chunk b (HALVES), or the neighbours within each.
template <bool HALVES>
__device__ __forceinline__ void turn(u32x4& a, u32x4& b, const double2 (&cs)[8]) {
  auto one = [](uint32_t lo, uint32_t hi, double2 t) {  // (x1, x2) as BF16 bits -> two of them
    const double x1 = bf16_to_f32(lo), x2 = bf16_to_f32(hi);
    v2f32k f;
    f[0] = (float)__builtin_fma(x1, t.x, -(x2 * t.y));
    f[1] = (float)__builtin_fma(x2, t.x, x1 * t.y);
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2k));
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (HALVES) {
      const uint32_t u = one(a[i] & 0xFFFFu, b[i] & 0xFFFFu, cs[2 * i]);
      const uint32_t v = one(a[i] >> 16, b[i] >> 16, cs[2 * i + 1]);
      a[i] = (u & 0xFFFFu) | (v << 16);
      b[i] = (u >> 16) | (v & 0xFFFF0000u);
    } else {
      a[i] = one(a[i] & 0xFFFFu, a[i] >> 16, cs[i]);
      b[i] = one(b[i] & 0xFFFFu, b[i] >> 16, cs[4 + i]);
    }
  }
}

template <int FMT, int D, bool HALVES>
__global__ __launch_bounds__(KV_THREADS) void k_kv_append_rotated(RotArgs p) {
  typedef KvLayout<FMT, D> L;
  constexpr int ITEMS = D / 16, HEADS = 64 / ITEMS, WAVES = KV_THREADS / 64;
  __shared__ double2 s_cs[WAVES][D / 2];
  __shared__ u32x4 s_k[WAVES][HEADS * D / 8];
  __shared__ u32x4 s_v[WAVES][32];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const KvArgs& c = p.kv;
  const int64_t row = (int64_t)blockIdx.x * WAVES + wave;
  if (row >= c.rows) return;

  // this lane's chunks of a head; the first heads' loads are on their way while the
  // token's place is looked up
  const int item = lane % ITEMS, h0 = lane / ITEMS;
  const bool pair = item < p.half / 8;
  const int c1 = HALVES && pair ? 8 * item : 16 * item;
  const int c2 = HALVES && pair ? p.half + 8 * item : 16 * item + 8;
  const bool with_q = p.per == 0 || blockIdx.y > 0, with_kv = p.per == 0 || blockIdx.y == 0;
  const int from = p.per == 0 ? 0 : ((int)blockIdx.y - 1) * p.per;
  const int to = p.per == 0 ? p.heads : min(p.heads, from + p.per);
  const uint16_t* const qs = p.q + row * p.ldq;
  const uint16_t* const ks = c.k + row * c.ldk;
  u32x4 q1, q2, k1, k2;
  if (with_q && from + h0 < to) {
    q1 = *reinterpret_cast<const u32x4*>(qs + (from + h0) * D + c1);
    q2 = *reinterpret_cast<const u32x4*>(qs + (from + h0) * D + c2);
  }
  if (with_kv && h0 < c.H) {
    k1 = *reinterpret_cast<const u32x4*>(ks + h0 * D + c1);
    k2 = *reinterpret_cast<const u32x4*>(ks + h0 * D + c2);
  }

  // where the token stands (of no sequence: its q is copied, nothing is stored)
  const bool on = row >= c.off[0] && row < c.off[c.B];
  uint8_t* page_of = nullptr;
  int slot = 0;
  if (on) {
    const WaveSequence sq = wave_sequence(c, row, lane);
    const int64_t pos = (int64_t)sq.len - sq.end + row;
    const int64_t at = p.positions ? (int64_t)p.positions[row] : pos;
    const int64_t pg = pos >> c.page_shift;
    int64_t id = -1;
    if (with_kv && pos >= 0 && pg < c.table_cols) id = c.table[sq.b * c.ldt + pg];
    for (int i = lane; i < p.half; i += 64) s_cs[wave][i] = cos_sin((double)at * (double)p.freqs[i]);
    if (id >= 0 && id < c.n_pages) {
      const int page = 1 << c.page_shift;
      slot = (int)(pos & (page - 1));
      page_of = c.cache + id * c.H * (int64_t)L::bytes(page);
    }
  }
  wave_fence();

  const bool turns = on && pair;
  double2 cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = turns ? s_cs[wave][8 * item + i] : make_double2(1.0, 0.0);

  if (with_q) {
    uint16_t* const dst = p.qo + row * p.ldqo;
    for (int h = from + h0; h < to; h += HEADS) {
      if (h > from + h0) {
        q1 = *reinterpret_cast<const u32x4*>(qs + h * D + c1);
        q2 = *reinterpret_cast<const u32x4*>(qs + h * D + c2);
      }
      if (turns) turn<HALVES>(q1, q2, cs);
      *reinterpret_cast<u32x4*>(dst + h * D + c1) = q1;
      *reinterpret_cast<u32x4*>(dst + h * D + c2) = q2;
    }
  }
  if (!with_kv || page_of == nullptr) return;

  // keys: by HEADS heads into LDS, from there 32 elements to each of the lower
  // lanes; the upper ones quantize the same heads' values
  const int page = 1 << c.page_shift, run = lane & 31, j = run % L::J;
  const bool is_v = lane >= 32;
  for (int hb = 0; hb < c.H; hb += HEADS) {
    const int h = hb + h0, hq = hb + run / L::J;
    if (h < c.H) {
      if (hb > 0) {
        k1 = *reinterpret_cast<const u32x4*>(ks + h * D + c1);
        k2 = *reinterpret_cast<const u32x4*>(ks + h * D + c2);
      }
      if (turns) turn<HALVES>(k1, k2, cs);
      s_k[wave][(h0 * D + c1) / 8] = k1;
      s_k[wave][(h0 * D + c2) / 8] = k2;
    }
    wave_fence();
    if (hq < c.H) {
      uint32_t x[16], w[4], s;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x4 u = is_v ? reinterpret_cast<const u32x4*>(c.v + row * c.ldv + hq * D + j * 32)[i]
                             : s_k[wave][run * 4 + i];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * i + e] = u[e];
      }
      const float t = FMT == FP4Q_NVFP4 ? (is_v ? c.vts : c.kts)[hq] : 1.0f;
      quant32<FMT>(x, t, w, s);
      uint8_t* base = page_of + hq * (int64_t)L::bytes(page);
      store_scales<FMT, D>(base, is_v, page, slot, j, s);
      if (!is_v) {
        store_k<FMT, D>(base, slot, j, w);
      } else {
        const u32x4 b = v_bytes_from_codes<L::J>(w, j, reinterpret_cast<uint8_t*>(s_v[wave]) + run / L::J * (16 * L::J));
        store_v<FMT, D>(base, page, slot, j, b);
      }
    }
    wave_fence();
  }
}

template <int FMT, int D>
void launch(bool append, const KvArgs& p, hipStream_t stream) {
  const int64_t items = (p.rows + 3) / 4 * 4 * p.H * (D / 32);
  const dim3 grid((unsigned)((items + KV_THREADS - 1) / KV_THREADS), 2);
  if (append) hipLaunchKernelGGL((k_kv_append<FMT, D>), grid, dim3(KV_THREADS), 0, stream, p);
  else hipLaunchKernelGGL((k_kv_read<FMT, D>), grid, dim3(KV_THREADS), 0, stream, p);
}

template <int FMT, int D>
void launch_rotated(const RotArgs& p, hipStream_t stream) {
  const int64_t blocks = (p.kv.rows + 3) / 4;
  const dim3 grid((unsigned)blocks, p.per == 0 ? 1u : (unsigned)(1 + (p.heads + p.per - 1) / p.per));
  if (p.halves) hipLaunchKernelGGL((k_kv_append_rotated<FMT, D, true>), grid, dim3(KV_THREADS), 0, stream, p);
  else hipLaunchKernelGGL((k_kv_append_rotated<FMT, D, false>), grid, dim3(KV_THREADS), 0, stream, p);
}

}  // namespace

void launch_kv_append_rotated(int fmt, uint8_t* cache, int64_t n_pages, int page_shift, int H, int D,
                              const int32_t* off, int B, const int32_t* table, int64_t ldt,
                              int64_t table_cols, const int32_t* lens, int64_t rows, const uint16_t* q,
                              int64_t ldq, int heads, uint16_t* qo, int64_t ldqo, const uint16_t* k,
                              int64_t ldk, const uint16_t* v, int64_t ldv, const float* freqs, int half,
                              bool halves, const int32_t* positions, const float* kts, const float* vts,
                              hipStream_t stream) {
  RotArgs p = {};
  p.kv = {cache, n_pages, page_shift, H, off, B, table, ldt, table_cols, lens, rows,
          const_cast<uint16_t*>(k), const_cast<uint16_t*>(v), ldk, ldv, kts, vts};
  p.q = q;
  p.qo = qo;
  p.ldq = ldq;
  p.ldqo = ldqo;
  p.heads = heads;
  p.half = half;
  p.halves = halves;
  p.freqs = freqs;
  p.positions = positions;
  // Few tokens: their heads over several workgroups, each with its own sines (us of
  // NVFP4, 32 + 8 heads of 128, with and without: 1 row 5.4 and 7.1, 64 6.2 and 8.1, 1024
  // 9.6 and 11.2, 1536 11.9 and 12.8, 2048 14.2 and 13.6, 8192 48.6 and 41.6).
  const int once = 64 / (D / 16);  // heads that a wave has at a time
  p.per = rows <= 1536 && heads > once ? once : 0;
  if (p.per > 0 && (heads + p.per - 1) / p.per > 65534) p.per = 0;
  if (fmt == FP4Q_NVFP4) {
    if (D == 64) launch_rotated<FP4Q_NVFP4, 64>(p, stream);
    else if (D == 128) launch_rotated<FP4Q_NVFP4, 128>(p, stream);
    else launch_rotated<FP4Q_NVFP4, 256>(p, stream);
  } else {
    if (D == 64) launch_rotated<FP4Q_MXFP4, 64>(p, stream);
    else if (D == 128) launch_rotated<FP4Q_MXFP4, 128>(p, stream);
    else launch_rotated<FP4Q_MXFP4, 256>(p, stream);
  }
}

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
