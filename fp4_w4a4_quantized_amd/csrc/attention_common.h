// attention_common.h -- what the kernels of attention over the paged FP4
// key/value cache have in common: the call's arguments, the keys a tile of
// rows sees, and the exact decoding of the cache's bytes.
#pragma once
#include "fp4q_device.h"
#include "fp4q_internal.h"
#include "kv_layout.h"

namespace fp4q {

struct AttnArgs {
  const uint8_t* cache;
  int64_t n_pages;
  int page_shift, H, G;
  const int32_t* off;
  int B;
  const int32_t* table;
  int64_t ldt;
  int cap;  // keys from here on are not seen: the table's end, or max_len
  const int32_t* lens;
  const uint16_t* q;
  int64_t ldq;
  int rows;
  int max_new;  // new tokens of a sequence that are attended for (further ones give 0)
  int window;
  float scale2;  // softmax scale * log2(e)
  const float* kts;
  const float* vts;
  void* y;
  int64_t ldy;
  int y_bf16;
  int chunk;   // keys of a split (a multiple of step)
  int splits;  // splits launched; 1: the kernel writes y itself
  int tile;    // rows of a workgroup
  int step;    // keys of a step of its kernel: splits begin at its multiples
  int join;    // groups of lanes that join a row's splits
  int64_t slots;  // rows * heads: partial results of one split
  float2* part_ms;  // [splits][slots] (maximum in log2 units, a whole number; sum)
  float* part_o;    // [splits][slots][D]
};

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef uint32_t w4 __attribute__((ext_vector_type(4)));

constexpr float P_BIAS = 7.0f;   // log2 of p at the running maximum
constexpr float P_SLACK = 8.0f;  // the maximum may fall behind by 2^8: p <= 2^15
// Products' factor to log2 units, at least: a masked one, -inf, times it stays -inf.
constexpr float MIN_FACTOR = 0x1p-149f;
constexpr int ROWS = 16;         // rows of a wave (columns of its products)
constexpr int KEYS = 32;         // keys of a step

// Keys [seen, hi) that some row of the tile sees (none if there are none
// left), lo: seen brought down to a step's boundary.
struct Range {
  int64_t r0;       // first new-token row of the sequence
  int n, first;     // new tokens, position of the first (below 0 if there are too many)
  int seen, lo, hi, rows;
};

// New-token rows of sequence b times the heads of a kv head (none past max_new,
// and none that the packed tensors do not have, whatever the offsets say).
__device__ __forceinline__ int tile_rows(const AttnArgs& p, int b) {
  const int r0 = p.off[b], r1 = min(p.off[b + 1], p.rows);
  return r0 < 0 || r1 <= r0 ? 0 : min(r1 - r0, p.max_new) * p.G;
}

// The first key that the row at position pos sees (pos may be below 0, the
// window up to 2^31 - 1: their difference would wrap).
__device__ __forceinline__ int first_key(const AttnArgs& p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

__device__ __forceinline__ Range tile_range(const AttnArgs& p, int b, int row0) {
  Range r;
  r.r0 = p.off[b];
  r.n = p.off[b + 1] - p.off[b];
  const int len = min(max(p.lens[b], 0), p.cap);
  r.first = p.lens[b] - r.n;
  r.rows = tile_rows(p, b);
  const int last_row = min(r.rows, row0 + p.tile) - 1;
  const int q_lo = row0 / p.G, q_hi = last_row / p.G;
  r.hi = min(len, r.first + q_hi + 1);
  r.seen = first_key(p, r.first + q_lo);
  // (never past the keys that there are: the waves count on from it)
  r.lo = min(r.seen, max(r.hi, 0)) & ~(p.step - 1);
  return r;
}

// Splits of the tile's keys, and where one that begins at k0 ends.
__device__ __forceinline__ int active_splits(const AttnArgs& p, const Range& r) {
  const int keys = r.hi - r.lo;
  return keys > 0 ? (keys - 1) / p.chunk + 1 : 1;  // (keys + chunk may pass 2^31)
}

__device__ __forceinline__ int split_end(const AttnArgs& p, const Range& r, int k0) {
  return r.hi - k0 > p.chunk ? k0 + p.chunk : r.hi;
}

template <int FMT> struct Num;
template <> struct Num<FP4Q_NVFP4> {
  typedef h8 vec;
  typedef h2 pair;
  static __device__ __forceinline__ v4f mfma(vec a, vec b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <> struct Num<FP4Q_MXFP4> {
  typedef b8 vec;
  typedef b2 pair;
  static __device__ __forceinline__ v4f mfma(vec a, vec b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

// Two codes (byte SEL of w) times their scale(s), exact.  NVFP4: s holds both
// scales as f16; MXFP4: e8 is the block's scale as a float.
template <int SEL>
__device__ __forceinline__ h2 decode2(uint32_t w, h2 s) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL) * s;
}
template <int SEL>
__device__ __forceinline__ b2 decode2(uint32_t w, float e8) {
  return __builtin_bit_cast(b2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, e8, SEL));
}

__device__ __forceinline__ h2 e4m3_pair(uint32_t w, int half) {
  return half ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)
              : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
}

__device__ __forceinline__ uint32_t as_u32(h2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ uint32_t as_u32(b2 v) { return __builtin_bit_cast(uint32_t, v); }

// One 16-key subtile as loaded: lane (c, g) holds the K bytes of key c,
// elements g D/4 ..; the V bytes of keys 4g .. 4g+3, elements c, c + 16, ...;
// its K scales (low bytes of ks) and the V scales of its four keys.
template <int FMT, int D>
struct Sub {
  typedef KvLayout<FMT, D> L;
  static constexpr int KW = D / 32;  // dwords of codes
  static constexpr int VS = L::SB;   // dwords of V scales (4 tokens)
  uint32_t k[KW], v[KW], ks, vs[VS];
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const w4 u = reinterpret_cast<const w4*>(p)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * i + e] = u[e];
    }
  } else {
    static_assert(N == 2, "");
    const u32x2 u = *reinterpret_cast<const u32x2*>(p);
    w[0] = u[0];
    w[1] = u[1];
  }
}

// Loads through a buffer descriptor: the address is scalar but for one 32-bit
// offset a lane, where plain loads would keep 64-bit vector addresses.
typedef __amdgpu_buffer_rsrc_t Buffer;

__device__ __forceinline__ Buffer page_buffer(const uint8_t* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes, 0x00027000);
}

template <int N>
__device__ __forceinline__ void buffer_words(Buffer r, uint32_t lane_off, uint32_t off, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const w4 u = __builtin_bit_cast(w4, __builtin_amdgcn_raw_buffer_load_b128(r, lane_off + 16 * i, off, 0));
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * i + e] = u[e];
    }
  } else {
    static_assert(N == 2, "");
    const u32x2 u = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, lane_off, off, 0));
    w[0] = u[0];
    w[1] = u[1];
  }
}

// The subtile that starts at `slot` of a page of one head.
template <int FMT, int D>
__device__ __forceinline__ void load_k(Buffer r, int page, int slot, int lane, Sub<FMT, D>& s) {
  typedef KvLayout<FMT, D> L;
  const uint32_t c = lane & 15, g = lane >> 4;
  buffer_words(r, c * (D / 2) + g * (D / 8), slot * (D / 2), s.k);
  constexpr int KS = L::SB >= 4 ? L::SB / 4 : 1;  // scale bytes of a lane (two lanes: one)
  const uint32_t at = c * L::SB + (L::SB >= 4 ? g * KS : g >> 1), off = L::k_scales(page) + slot * L::SB;
  if constexpr (KS == 1) s.ks = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, at, off, 0);
  else if constexpr (KS == 2) s.ks = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, off, 0);
  else s.ks = __builtin_amdgcn_raw_buffer_load_b32(r, at, off, 0);
}

template <int FMT, int D>
__device__ __forceinline__ void load_v(Buffer r, int page, int slot, int lane, Sub<FMT, D>& s) {
  typedef KvLayout<FMT, D> L;
  buffer_words(r, lane * (D / 8), L::v_codes(page) + slot * (D / 2), s.v);
  buffer_words(r, (lane >> 4) * 4 * L::SB, L::v_scales(page) + slot * L::SB, s.vs);
}

// A K block's scale as decode2 takes it: the low byte(s) of s hold its code
// (NVFP4: blk 0 or 1 of two).
template <int FMT>
__device__ __forceinline__ auto k_scale(uint32_t s, int blk) {
  if constexpr (FMT == FP4Q_NVFP4) {
    const h2 both = e4m3_pair(s, 0);
    const _Float16 e = blk ? both[1] : both[0];
    return h2{e, e};
  } else {
    return __uint_as_float((s & 0xFFu) << 23);
  }
}

// The eight values of a dword of K codes.
template <int FMT, typename Scale>
__device__ __forceinline__ typename Num<FMT>::vec decode8(uint32_t w, Scale sc) {
  w4 r;
  r[0] = as_u32(decode2<0>(w, sc));
  r[1] = as_u32(decode2<1>(w, sc));
  r[2] = as_u32(decode2<2>(w, sc));
  r[3] = as_u32(decode2<3>(w, sc));
  return __builtin_bit_cast(typename Num<FMT>::vec, r);
}

// K operand of step st (8 elements: dword st of the lane's codes).
template <int FMT, int D>
__device__ __forceinline__ typename Num<FMT>::vec decode_k(const Sub<FMT, D>& s, int st) {
  if constexpr (FMT == FP4Q_NVFP4)  // a lane's dwords: two to a block
    return decode8<FMT>(s.k[st], k_scale<FMT>(s.ks >> (16 * (st >> 2)), (st >> 1) & 1));
  else
    return decode8<FMT>(s.k[st], k_scale<FMT>(s.ks >> (8 * (st >> 2)), 0));
}

// The values of token t (0..3), elements (32j + c, 32j + 16 + c).
template <int FMT, int D, int T, int JJ>
__device__ __forceinline__ uint32_t decode_v(const Sub<FMT, D>& s) {
  constexpr int J = D / 32, byte = T * J + JJ;
  const uint32_t w = s.v[byte >> 2];
  if constexpr (FMT == FP4Q_NVFP4) {
    constexpr int hw = byte;  // halfword: scales 2j, 2j + 1 of the token
    return as_u32(decode2<(byte & 3)>(w, e4m3_pair(s.vs[hw >> 1], hw & 1)));
  } else {
    // (scales above 2^125 count as 2^125: every value is finite, so that a
    // weight of 0 removes it)
    const uint32_t e = min((s.vs[byte >> 2] >> (8 * (byte & 3))) & 0xFFu, 252u);
    return as_u32(decode2<(byte & 3)>(w, __uint_as_float(e << 23)));
  }
}

// Run JJ of the four tokens: their elements 32 JJ + c (lo) and 32 JJ + 16 + c
// (hi), two tokens to a dword.
template <int FMT, int D, int JJ>
__device__ __forceinline__ void v_run(const Sub<FMT, D>& s, u32x2& lo, u32x2& hi) {
  const uint32_t a0 = decode_v<FMT, D, 0, JJ>(s), a1 = decode_v<FMT, D, 1, JJ>(s),
                 a2 = decode_v<FMT, D, 2, JJ>(s), a3 = decode_v<FMT, D, 3, JJ>(s);
  // v_perm_b32: bytes 0-3 from the second operand, 4-7 from the first
  lo[0] = __builtin_amdgcn_perm(a1, a0, 0x05040100u);
  lo[1] = __builtin_amdgcn_perm(a3, a2, 0x05040100u);
  hi[0] = __builtin_amdgcn_perm(a1, a0, 0x07060302u);
  hi[1] = __builtin_amdgcn_perm(a3, a2, 0x07060302u);
}

template <int FMT, int D, int JJ, typename F>
__device__ __forceinline__ void v_rows(const Sub<FMT, D>& s, F f) {
  u32x2 lo, hi;
  v_run<FMT, D, JJ>(s, lo, hi);
  f(JJ, lo, hi);
  if constexpr (JJ + 1 < D / 32) v_rows<FMT, D, JJ + 1>(s, f);
}

// The V scales of tokens key .. key + 3 outside [seen, hi) become 0 (all of
// them where the page is not in the cache): what stands there may be
// anything, and a weight of 0 would not remove a NaN.
template <int FMT, int D>
__device__ __forceinline__ void zero_v_scales(Sub<FMT, D>& s, int key, bool all, int seen, int hi) {
  constexpr int SB = KvLayout<FMT, D>::SB;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (!all && key + t >= seen && key + t < hi) continue;
#pragma unroll
    for (int i = 0; i < Sub<FMT, D>::VS; ++i) {
      uint32_t keep = 0xFFFFFFFFu;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((4 * i + e) / SB == t) keep &= ~(0xFFu << (8 * e));
      s.vs[i] &= keep;
    }
  }
}

// O^T tiles 2j and 2j + 1 (elements 32j + .. and 32j + 16 + ..) += V^T P^T.
template <int FMT, int D, int JJ, int NC>
__device__ __forceinline__ void pv(const Sub<FMT, D>& s0, const Sub<FMT, D>& s1,
                                   const typename Num<FMT>::vec (&pb)[NC], v4f (&o)[NC][D / 16]) {
  typedef typename Num<FMT>::vec vec;
  u32x2 l0, h0, l1, h1;
  v_run<FMT, D, JJ>(s0, l0, h0);
  v_run<FMT, D, JJ>(s1, l1, h1);
  const w4 lo = {l0[0], l0[1], l1[0], l1[1]}, hi = {h0[0], h0[1], h1[0], h1[1]};
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    o[n][2 * JJ] = Num<FMT>::mfma(__builtin_bit_cast(vec, lo), pb[n], o[n][2 * JJ]);
    o[n][2 * JJ + 1] = Num<FMT>::mfma(__builtin_bit_cast(vec, hi), pb[n], o[n][2 * JJ + 1]);
  }
}

template <int FMT, int D, int JJ, int NC>
__device__ __forceinline__ void pv_all(const Sub<FMT, D>& s0, const Sub<FMT, D>& s1,
                                       const typename Num<FMT>::vec (&pb)[NC],
                                       v4f (&o)[NC][D / 16]) {
  pv<FMT, D, JJ, NC>(s0, s1, pb, o);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (JJ + 1 < D / 32) pv_all<FMT, D, JJ + 1, NC>(s0, s1, pb, o);
}

// Maxima over the lanes 32 apart, and 16 apart.
__device__ __forceinline__ float other_half_max(float v) {
  const u32x2 r = __builtin_bit_cast(
      u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other_quarter_max(float v) {
  const u32x2 r = __builtin_bit_cast(
      u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ uint32_t max_magnitude(w4 u) {  // of 8 BF16, as bits
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) m = max(m, max(u[e] & 0x7FFFu, (u[e] >> 16) & 0x7FFFu));
  return m;
}

// The power of two that a row of q is divided by for f16: the exponent of its
// largest magnitude, held to where it and its reciprocal are normal numbers
// (infinities and NaN stay what they are).
__device__ __forceinline__ int q_exponent(uint32_t m) {
  return min(max((int)(m >> 7), 1), 253) - 127;
}

__device__ __forceinline__ w4 q_to_f16(w4 u, int sh) {
  const float down = __uint_as_float((uint32_t)(127 - sh) << 23);
  w4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v2f f = {__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xFFFF0000u)};
    f[0] *= down;
    f[1] *= down;
    r[e] = as_u32(__builtin_convertvector(f, h2));
  }
  return r;
}

// A row's operand: D/4 elements of q per lane in steps of 8, and its factor
// from products to log2 units.
template <int FMT, int D>
__device__ __forceinline__ void load_q(const uint16_t* q, int g, float c0,
                                       typename Num<FMT>::vec (&out)[D / 32], float& c) {
  typedef typename Num<FMT>::vec vec;
  w4 u[D / 32];
#pragma unroll
  for (int st = 0; st < D / 32; ++st)
    u[st] = *reinterpret_cast<const w4*>(q + g * (D / 4) + st * 8);
  if constexpr (FMT == FP4Q_MXFP4) {
#pragma unroll
    for (int st = 0; st < D / 32; ++st) out[st] = __builtin_bit_cast(vec, u[st]);
    c = c0;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int st = 0; st < D / 32; ++st) m = max(m, max_magnitude(u[st]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    const int sh = q_exponent(m);
    c = c0 * __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
    for (int st = 0; st < D / 32; ++st) out[st] = __builtin_bit_cast(vec, q_to_f16(u[st], sh));
  }
  c = fmaxf(c, MIN_FACTOR);
}

// What a split leaves the join of its maximum m (c: to log2 units): a whole
// number near m c, and f = 2^(m c - number) for its sums.  (m c itself, rounded,
// would weigh the splits by 2^(m c 2^-24) apart.)
__device__ __forceinline__ float whole_max(float m, float c, float& f) {
  const float r = rintf(m * c);
  // (past 2^24 the number's own rounding; beyond 2^29 scores are not known to 2^32)
  const float e = fminf(fmaxf(__builtin_fmaf(m, c, -r), -32.0f), 32.0f);
  f = __builtin_amdgcn_exp2f(e);
  return r;
}

// Four neighbouring outputs, from element `at` of y.
__device__ __forceinline__ void store_out(const AttnArgs& p, int64_t at, v4f t) {
  if (p.y_bf16) {
    const v2f f0 = {t[0], t[1]}, f1 = {t[2], t[3]};
    u32x2 u;
    u[0] = as_u32(__builtin_convertvector(f0, b2));
    u[1] = as_u32(__builtin_convertvector(f1, b2));
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p.y) + at) = u;
  } else {
    *reinterpret_cast<v4f*>(reinterpret_cast<float*>(p.y) + at) = t;
  }
}

// Rows past the last sequence's and past max_new of a sequence give 0 (of one
// pass; the join does it otherwise): workgroup (b, h) takes every B-th of the
// first kind and b's of the second, for the heads of kv head h.
template <int D, int THREADS>
__device__ __forceinline__ void zero_rest(const AttnArgs& p, int b, int h) {
  if (p.splits > 1 || blockIdx.y > 0) return;
  auto zero = [&](int64_t row) {
    for (int i = threadIdx.x * 4; i < p.G * D; i += THREADS * 4)
      store_out(p, row * p.ldy + (int64_t)h * p.G * D + i, v4f{0.0f, 0.0f, 0.0f, 0.0f});
  };
  for (int64_t row = (int64_t)max(p.off[p.B], 0) + b; row < p.rows; row += p.B) zero(row);
  const int64_t end = min(p.off[b + 1], p.rows);
  for (int64_t row = (int64_t)max(p.off[b], 0) + p.max_new; row < end; ++row) zero(row);
}

}  // namespace

void launch_attention_tile(int fmt, int D, const AttnArgs& p, int tiles, int B, hipStream_t stream);

}  // namespace fp4q
