// attention.hip -- attention over the paged FP4 key/value cache (defined in
// include/fp4q.h): per new token i and head,
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - m_i),
// over the keys j of its sequence with j <= position(i) (and j > position(i)
// - window), in one pass over the keys with a running maximum and sum.
//
// The heads that share a key/value head are rows of the same product: row r
// of a sequence's (kv head) is query r / G, head r % G of the group.  A wave
// takes 16 rows as the columns of 16x16x32 matrix instructions and 32 keys at
// a time:
//   S^T = K Q^T  (keys are the rows: a lane holds, for one of its columns,
//                 keys 4g .. 4g+3 of each 16, g = lane / 16)
//   O^T += V^T P^T  (k = keys: a lane's own S^T values, rounded, are its
//                 P^T operand, no exchange between lanes)
// K bytes: a lane holds D/4 consecutive elements of one key (the order of k
// is free as long as Q has the same).  V bytes: the cache keeps four tokens'
// bytes of one d mod 16 together, so that a lane's load is the 4 keys x D/16
// values its V^T operand needs.
//
// NVFP4 is decoded to f16 (e2m1 * E4M3 has at most 6 significant bits and
// lies in f16's range: exact; the head's tensor scale is factored out), MXFP4
// to bf16 (e2m1 * 2^e: exact).  q enters as f16 after a power of two brings
// the row's largest magnitude into [1, 2) (its smaller elements then lose at
// most 2^-25 of the largest), or as the bf16 it is.  P is rounded once to the
// same type (off by at most 2^-11 or 2^-8 of each weight, unbiased); scores,
// maximum, sum and output are FP32.  With f16, p is held 2^7 above the usual
// 2^(x - m), so that weights down to 2^-31 of the largest are not lost.
#include "fp4q_device.h"
#include "fp4q_internal.h"
#include "kv_layout.h"

namespace fp4q {

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
constexpr int ROWS = 16;         // rows of a wave (columns of its products)
constexpr int KEYS = 32;         // keys of a step

struct AttnArgs {
  const uint8_t* cache;
  int64_t n_pages;
  int page_shift, H, G;
  const int32_t* off;
  int B;
  const int32_t* table;
  int64_t ldt, table_cols;
  const int32_t* lens;
  const uint16_t* q;
  int64_t ldq;
  int window;
  float scale2;  // softmax scale * log2(e)
  const float* kts;
  const float* vts;
  void* y;
  int64_t ldy;
  int y_bf16;
  int chunk;   // keys of a split (a multiple of KEYS)
  int splits;  // splits launched; 1: the kernel writes y itself
  int tile;    // rows of a workgroup
  int64_t slots;  // rows * heads: partial results of one split
  float2* part_ms;  // [splits][slots] (maximum in log2 units, sum)
  float* part_o;    // [splits][slots][D]
};

// Keys [seen, hi) that some row of the tile sees (none if there are none
// left), lo: seen brought down to a step's boundary.
struct Range {
  int64_t r0;       // first new-token row of the sequence
  int n, first;     // new tokens, position of the first (below 0 if there are too many)
  int seen, lo, hi, rows;
};

__device__ __forceinline__ Range tile_range(const AttnArgs& p, int b, int row0) {
  Range r;
  r.r0 = p.off[b];
  r.n = p.off[b + 1] - p.off[b];
  const int64_t cap = p.table_cols << p.page_shift;
  const int len = (int)min((int64_t)max(p.lens[b], 0), cap);
  r.first = p.lens[b] - r.n;
  r.rows = r.n * p.G;
  const int last_row = min(r.rows, row0 + p.tile) - 1;
  const int q_lo = row0 / p.G, q_hi = last_row / p.G;
  r.hi = min(len, r.first + q_hi + 1);
  r.seen = p.window > 0 ? max(0, r.first + q_lo - p.window + 1) : 0;
  r.lo = r.seen & ~(KEYS - 1);
  return r;
}

__device__ __forceinline__ int active_splits(const AttnArgs& p, const Range& r) {
  const int keys = r.hi - r.lo;
  return keys > 0 ? (keys + p.chunk - 1) / p.chunk : 1;
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

// Loads of the subtile that starts at `slot` of a page (base: its bytes for
// this head).
template <int FMT, int D>
__device__ __forceinline__ void load_sub(const uint8_t* base, int page, int slot, int lane,
                                         Sub<FMT, D>& s) {
  typedef KvLayout<FMT, D> L;
  const int c = lane & 15, g = lane >> 4;
  load_words(base + slot * (D / 2) + c * (D / 2) + g * (D / 8), s.k);
  load_words(base + L::v_codes(page) + slot * (D / 2) + lane * (D / 8), s.v);
  const uint8_t* ks = base + L::k_scales(page) + (slot + c) * L::SB;
  if constexpr (FMT == FP4Q_NVFP4) {
    if constexpr (D == 64) s.ks = ks[g];
    else if constexpr (D == 128) s.ks = reinterpret_cast<const uint16_t*>(ks)[g];
    else s.ks = reinterpret_cast<const uint32_t*>(ks)[g];
  } else {
    if constexpr (D == 64) s.ks = ks[g >> 1];
    else if constexpr (D == 128) s.ks = ks[g];
    else s.ks = reinterpret_cast<const uint16_t*>(ks)[g];
  }
  load_words(base + L::v_scales(page) + (slot + 4 * g) * L::SB, s.vs);
}

// K operand of step st (8 elements: dword st of the lane's codes).
template <int FMT, int D>
__device__ __forceinline__ typename Num<FMT>::vec decode_k(const Sub<FMT, D>& s, int st) {
  typedef typename Num<FMT>::vec vec;
  w4 r;
  const uint32_t w = s.k[st];
  if constexpr (FMT == FP4Q_NVFP4) {
    const h2 both = e4m3_pair(s.ks >> (16 * (st >> 2)), 0);  // blocks 2(st/4), 2(st/4) + 1
    const _Float16 e = (st & 2) ? both[1] : both[0];
    const h2 sc = {e, e};
    r[0] = as_u32(decode2<0>(w, sc));
    r[1] = as_u32(decode2<1>(w, sc));
    r[2] = as_u32(decode2<2>(w, sc));
    r[3] = as_u32(decode2<3>(w, sc));
  } else {
    const float e8 = __uint_as_float(((s.ks >> (8 * (st >> 2))) & 0xFFu) << 23);
    r[0] = as_u32(decode2<0>(w, e8));
    r[1] = as_u32(decode2<1>(w, e8));
    r[2] = as_u32(decode2<2>(w, e8));
    r[3] = as_u32(decode2<3>(w, e8));
  }
  return __builtin_bit_cast(vec, r);
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
    const float e8 = __uint_as_float(((s.vs[byte >> 2] >> (8 * (byte & 3))) & 0xFFu) << 23);
    return as_u32(decode2<(byte & 3)>(w, e8));
  }
}

// O^T tiles 2j and 2j + 1 (elements 32j + .. and 32j + 16 + ..) += V^T P^T.
template <int FMT, int D, int JJ, int NC>
__device__ __forceinline__ void pv(const Sub<FMT, D>& s0, const Sub<FMT, D>& s1,
                                   const typename Num<FMT>::vec (&pb)[NC], v4f (&o)[NC][D / 16]) {
  typedef typename Num<FMT>::vec vec;
  const uint32_t a0 = decode_v<FMT, D, 0, JJ>(s0), a1 = decode_v<FMT, D, 1, JJ>(s0),
                 a2 = decode_v<FMT, D, 2, JJ>(s0), a3 = decode_v<FMT, D, 3, JJ>(s0);
  const uint32_t c0 = decode_v<FMT, D, 0, JJ>(s1), c1 = decode_v<FMT, D, 1, JJ>(s1),
                 c2 = decode_v<FMT, D, 2, JJ>(s1), c3 = decode_v<FMT, D, 3, JJ>(s1);
  w4 lo, hi;  // v_perm_b32: bytes 0-3 from the second operand, 4-7 from the first
  lo[0] = __builtin_amdgcn_perm(a1, a0, 0x05040100u);
  lo[1] = __builtin_amdgcn_perm(a3, a2, 0x05040100u);
  lo[2] = __builtin_amdgcn_perm(c1, c0, 0x05040100u);
  lo[3] = __builtin_amdgcn_perm(c3, c2, 0x05040100u);
  hi[0] = __builtin_amdgcn_perm(a1, a0, 0x07060302u);
  hi[1] = __builtin_amdgcn_perm(a3, a2, 0x07060302u);
  hi[2] = __builtin_amdgcn_perm(c1, c0, 0x07060302u);
  hi[3] = __builtin_amdgcn_perm(c3, c2, 0x07060302u);
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
  if constexpr (JJ + 1 < D / 32) pv_all<FMT, D, JJ + 1, NC>(s0, s1, pb, o);
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
    for (int st = 0; st < D / 32; ++st)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max(m, max(u[st][e] & 0x7FFFu, (u[st][e] >> 16) & 0x7FFFu));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    // 2^-s and 2^s, s the exponent of the largest magnitude (BF16 subnormals
    // and zero: left as they are)
    const int ex = (int)(m >> 7);
    const int sh = ex == 0 || ex >= 254 ? 0 : ex - 127;
    const float down = __uint_as_float((uint32_t)(127 - sh) << 23);
    c = c0 * __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
    for (int st = 0; st < D / 32; ++st) {
      w4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v2f f = {__uint_as_float(u[st][e] << 16), __uint_as_float(u[st][e] & 0xFFFF0000u)};
        f[0] *= down;
        f[1] *= down;
        r[e] = as_u32(__builtin_convertvector(f, h2));
      }
      out[st] = __builtin_bit_cast(vec, r);
    }
  }
  c = fmaxf(c, 1e-37f);  // (a masked product, -inf, times c stays -inf)
}

// WAVES waves share the keys of a (sequence, kv head, rows, split): wave w
// takes steps w, w + WAVES, ...
template <int FMT, int D, int NC, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_attn_split(AttnArgs p) {
  typedef typename Num<FMT>::vec vec;
  typedef typename Num<FMT>::pair pair;
  typedef KvLayout<FMT, D> L;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.z, h = blockIdx.y % p.H, row0 = (int)(blockIdx.y / p.H) * p.tile;
  const int n_rows = (p.off[b + 1] - p.off[b]) * p.G;
  if (row0 >= n_rows) return;
  const Range rg = tile_range(p, b, row0);
  const int split = blockIdx.x;
  if (split >= active_splits(p, rg)) return;
  const int k0 = rg.lo + split * p.chunk;
  const int k1 = min(rg.hi, k0 + p.chunk);

  vec qf[NC][D / 32];
  float cf[NC], m[NC], z[NC];
  int see_lo[NC], see_hi[NC];  // keys the column sees: [see_lo, see_hi)
  int64_t slot[NC];
  v4f o[NC][D / 16];
  int all_lo = 0, all_hi = 0x7FFFFFFF;
  const float c0 = p.scale2 * (FMT == FP4Q_NVFP4 ? p.kts[h] : 1.0f);
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int row = row0 + n * ROWS + c;
    const int rr = min(row, rg.rows - 1);
    const int qi = rr / p.G, hh = h * p.G + (rr - qi * p.G);
    load_q<FMT, D>(p.q + (rg.r0 + qi) * p.ldq + hh * D, g, c0, qf[n], cf[n]);
    see_hi[n] = min(rg.hi, rg.first + qi + 1);
    see_lo[n] = p.window > 0 ? rg.first + qi - p.window + 1 : 0;
    slot[n] = row < rg.rows ? (rg.r0 + qi) * (int64_t)(p.H * p.G) + hh : -1;
    m[n] = -__builtin_inff();
    z[n] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[n][i] = {0.0f, 0.0f, 0.0f, 0.0f};
  }
  {  // a step inside [all_lo, all_hi) needs no mask
    const int last = min(rg.rows, row0 + p.tile) - 1;
    all_hi = rg.first + row0 / p.G + 1;
    all_lo = p.window > 0 ? rg.first + last / p.G - p.window + 1 : 0;
  }

  const int page = 1 << p.page_shift;
  const int32_t* table = p.table + b * p.ldt;
  for (int kt = k0 + wave * KEYS; kt < k1; kt += WAVES * KEYS) {
    Sub<FMT, D> s[2];
    bool good[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = kt + 16 * u;
      int64_t id = -1;
      if (key < rg.hi) id = table[key >> p.page_shift];
      good[u] = id >= 0 && id < p.n_pages;
      if (!good[u]) id = 0;  // some page's bytes, all masked
      load_sub<FMT, D>(p.cache + (id * p.H + h) * (int64_t)L::bytes(page), page,
                       key & (page - 1), lane, s[u]);
    }
    const bool whole = good[0] && good[1] && kt >= all_lo && kt + KEYS <= all_hi;
    if (!whole) {
      // scales of keys that no row sees may hold anything: 0 for NaN's sake
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int key = kt + 16 * u + 4 * g + t;
          if (good[u] && key >= rg.seen && key < rg.hi) continue;
          constexpr int SB = L::SB;
#pragma unroll
          for (int i = 0; i < Sub<FMT, D>::VS; ++i) {
            uint32_t keep = 0xFFFFFFFFu;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((4 * i + e) / SB == t) keep &= ~(0xFFu << (8 * e));
            s[u].vs[i] &= keep;
          }
        }
    }
    vec pb[NC];
    float up = 0.0f;  // does some column's maximum run ahead of its kept one?
    v4f x[NC][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int n = 0; n < NC; ++n) x[n][u] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < D / 32; ++st) {
        const vec a = decode_k<FMT, D>(s[u], st);
#pragma unroll
        for (int n = 0; n < NC; ++n) x[n][u] = Num<FMT>::mfma(a, qf[n][st], x[n][u]);
      }
    }
    float mt[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = kt + 16 * u + 4 * g + r;
            if (!good[u] || key < see_lo[n] || key >= see_hi[n]) x[n][u][r] = -__builtin_inff();
          }
      }
      float t = fmaxf(fmaxf(fmaxf(x[n][0][0], x[n][0][1]), fmaxf(x[n][0][2], x[n][0][3])),
                      fmaxf(fmaxf(x[n][1][0], x[n][1][1]), fmaxf(x[n][1][2], x[n][1][3])));
      t = fmaxf(t, __shfl_xor(t, 16));
      t = fmaxf(t, __shfl_xor(t, 32));
      mt[n] = fmaxf(t, m[n]);
      if (mt[n] > -__builtin_inff())
        up = fmaxf(up, m[n] > -__builtin_inff() ? (mt[n] - m[n]) * cf[n] : P_SLACK + 1.0f);
    }
    if (__any(up > P_SLACK)) {
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const float base = mt[n] > -__builtin_inff() ? mt[n] : 0.0f;
        const float f = __builtin_amdgcn_exp2f((m[n] - base) * cf[n]);  // 0 from -inf
        m[n] = mt[n];
        z[n] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[n][i][r] *= f;
      }
    }
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      // (the difference first: m c alone may be past what 32 bits hold to 2^8)
      const float base = m[n] > -__builtin_inff() ? m[n] : 0.0f;
      w4 pk;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          v2f e;
          e[0] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][u][r] - base, cf[n], P_BIAS));
          e[1] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][u][r + 1] - base, cf[n], P_BIAS));
          z[n] += e[0] + e[1];
          pk[2 * u + (r >> 1)] = as_u32(__builtin_convertvector(e, pair));
        }
      pb[n] = __builtin_bit_cast(vec, pk);
    }
    pv_all<FMT, D, 0, NC>(s[0], s[1], pb, o);
  }

  // the waves' results meet: common maximum, summed sums and outputs
  __shared__ float s_m[WAVES][NC * ROWS], s_z[WAVES][NC * ROWS];
  __shared__ float s_o[WAVES][ROWS][D + 4];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    z[n] += __shfl_xor(z[n], 16);
    z[n] += __shfl_xor(z[n], 32);
    if (g == 0) {
      s_m[wave][n * ROWS + c] = m[n] * cf[n];
      s_z[wave][n * ROWS + c] = z[n];
    }
  }
  __syncthreads();
  const float vt = FMT == FP4Q_NVFP4 ? p.vts[h] : 1.0f;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    float mm = -__builtin_inff(), zz = 0.0f;
    for (int w = 0; w < WAVES; ++w) mm = fmaxf(mm, s_m[w][n * ROWS + c]);
    const float base = mm > -__builtin_inff() ? mm : 0.0f;
    for (int w = 0; w < WAVES; ++w)
      zz += s_z[w][n * ROWS + c] * __builtin_amdgcn_exp2f(s_m[w][n * ROWS + c] - base);
    const float mine = __builtin_amdgcn_exp2f(m[n] * cf[n] - base);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      v4f t;
#pragma unroll
      for (int r = 0; r < 4; ++r) t[r] = o[n][i][r] * mine;
      *reinterpret_cast<v4f*>(&s_o[wave][c][16 * i + 4 * g]) = t;
    }
    __syncthreads();
    // thread: column c2, elements d, d + 4 * STEP, ...
    for (int i = threadIdx.x; i < ROWS * D / 4; i += 64 * WAVES) {
      const int col = i / (D / 4), d = (i - col * (D / 4)) * 4;
      const int row = row0 + n * ROWS + col;
      if (row >= rg.rows) continue;
      v4f t = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int w = 0; w < WAVES; ++w) {
        const v4f a = *reinterpret_cast<const v4f*>(&s_o[w][col][d]);
#pragma unroll
        for (int r = 0; r < 4; ++r) t[r] += a[r];
      }
      const int qi = row / p.G, hh = h * p.G + (row - qi * p.G);
      if (p.splits == 1) {
        float zc = 0.0f, mc = -__builtin_inff();
        for (int w = 0; w < WAVES; ++w) mc = fmaxf(mc, s_m[w][n * ROWS + col]);
        const float bc = mc > -__builtin_inff() ? mc : 0.0f;
        for (int w = 0; w < WAVES; ++w)
          zc += s_z[w][n * ROWS + col] * __builtin_amdgcn_exp2f(s_m[w][n * ROWS + col] - bc);
        const float f = zc > 0.0f ? vt / zc : 0.0f;
        const int64_t at = (rg.r0 + qi) * p.ldy + hh * D + d;
        if (p.y_bf16) {
          const v2f f0 = {t[0] * f, t[1] * f}, f1 = {t[2] * f, t[3] * f};
          u32x2 u;
          u[0] = as_u32(__builtin_convertvector(f0, b2));
          u[1] = as_u32(__builtin_convertvector(f1, b2));
          *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p.y) + at) = u;
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) t[r] *= f;
          *reinterpret_cast<v4f*>(reinterpret_cast<float*>(p.y) + at) = t;
        }
      } else {
        const int64_t s = split * p.slots + (rg.r0 + qi) * (int64_t)(p.H * p.G) + hh;
        *reinterpret_cast<v4f*>(p.part_o + s * D + d) = t;
      }
    }
    if (p.splits > 1 && wave == 0 && g == 0 && slot[n] >= 0)
      p.part_ms[split * p.slots + slot[n]] = make_float2(mm, zz);
    __syncthreads();
  }
}

// Joins the splits of a row: one wave per (new token, head).
template <int FMT, int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t s = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (s >= p.slots) return;
  const int heads = p.H * p.G;
  const int64_t row = s / heads;
  const int hh = (int)(s - row * heads);
  if (row < p.off[0] || row >= p.off[p.B]) return;
  const int b = kv_sequence(p.off, p.B, row);
  const int r = (int)(row - p.off[b]) * p.G + hh % p.G;
  const Range rg = tile_range(p, b, r / p.tile * p.tile);
  const int n = min(active_splits(p, rg), p.splits);
  float m = -__builtin_inff();
  for (int i = lane; i < n; i += 64) m = fmaxf(m, p.part_ms[i * p.slots + s].x);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float base = m > -__builtin_inff() ? m : 0.0f;
  float z = 0.0f, o[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) o[e] = 0.0f;
  for (int i = 0; i < n; ++i) {
    const float2 ms = p.part_ms[i * p.slots + s];
    const float f = __builtin_amdgcn_exp2f(ms.x - base);
    z += ms.y * f;
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
      o[e] = __builtin_fmaf(p.part_o[(i * p.slots + s) * D + e * 64 + lane], f, o[e]);
  }
  const float f = z > 0.0f ? (FMT == FP4Q_NVFP4 ? p.vts[hh / p.G] : 1.0f) / z : 0.0f;
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    const int64_t at = row * p.ldy + hh * D + e * 64 + lane;
    if (p.y_bf16) reinterpret_cast<__bf16*>(p.y)[at] = (__bf16)(o[e] * f);
    else reinterpret_cast<float*>(p.y)[at] = o[e] * f;
  }
}

// How a call is split: a function of host numbers only, so that the workspace
// query and the launch agree.
struct Plan {
  int nc, tile, tiles, chunk, splits;
};

Plan attn_plan(int D, int B, int H, int G, int64_t max_new, int64_t max_len, int window) {
  Plan p;
  const int64_t rows = max_new * G;
  p.nc = rows > ROWS && D <= 128 ? 2 : 1;
  p.tile = ROWS * p.nc;
  p.tiles = (int)((rows + p.tile - 1) / p.tile);
  int64_t keys = max_len;
  if (window > 0) keys = keys < window + max_new + KEYS ? keys : window + max_new + KEYS;
  // enough workgroups to fill the card a few times over, and at least 256 keys each
  const int64_t groups = (int64_t)B * H * p.tiles;
  int64_t chunk = (keys * groups + 2047) / 2048;
  chunk = chunk < 256 ? 256 : chunk;
  chunk = (chunk + KEYS - 1) / KEYS * KEYS;
  p.chunk = (int)(chunk < (1 << 30) ? chunk : (1 << 30));
  p.splits = (int)((keys + p.chunk - 1) / p.chunk);
  if (p.splits < 1) p.splits = 1;
  return p;
}

template <int FMT, int D>
void launch(const AttnArgs& p, const Plan& pl, int H, int B, hipStream_t stream) {
  const dim3 grid((unsigned)pl.splits, (unsigned)(H * pl.tiles), (unsigned)B), thr(256);
  if constexpr (D <= 128) {
    if (pl.nc == 2) hipLaunchKernelGGL((k_attn_split<FMT, D, 2, 4>), grid, thr, 0, stream, p);
    else hipLaunchKernelGGL((k_attn_split<FMT, D, 1, 4>), grid, thr, 0, stream, p);
  } else {
    hipLaunchKernelGGL((k_attn_split<FMT, D, 1, 4>), grid, thr, 0, stream, p);
  }
  if (pl.splits > 1)
    hipLaunchKernelGGL((k_attn_join<FMT, D>), dim3((unsigned)((p.slots + 3) / 4)), thr, 0, stream, p);
}

}  // namespace

bool attention_shape_ok(int D, int B, int H, int G, int64_t max_new, int64_t max_len, int window) {
  const Plan pl = attn_plan(D, B, H, G, max_new, max_len, window);
  return B <= 65535 && (int64_t)H * pl.tiles <= 65535;
}

size_t attention_workspace_bytes(int64_t rows, int D, int B, int H, int G, int64_t max_new,
                                 int64_t max_len, int window) {
  const Plan pl = attn_plan(D, B, H, G, max_new, max_len, window);
  return pl.splits > 1 ? (size_t)pl.splits * (size_t)(rows * H * G) * (size_t)(D + 2) * 4 : 0;
}

void launch_attention(int fmt, const uint8_t* cache, int64_t n_pages, int page_shift, int H, int D,
                      const int32_t* off, int B, const int32_t* table, int64_t ldt, int64_t table_cols,
                      const int32_t* lens, const uint16_t* q, int64_t ldq, int64_t rows, int G,
                      int64_t max_new, int64_t max_len, int window, float scale, const float* kts,
                      const float* vts, void* y, int y_bf16, int64_t ldy, void* ws,
                      hipStream_t stream) {
  const Plan pl = attn_plan(D, B, H, G, max_new, max_len, window);
  AttnArgs p = {};
  p.cache = cache;
  p.n_pages = n_pages;
  p.page_shift = page_shift;
  p.H = H;
  p.G = G;
  p.off = off;
  p.B = B;
  p.table = table;
  p.ldt = ldt;
  p.table_cols = table_cols;
  p.lens = lens;
  p.q = q;
  p.ldq = ldq;
  p.window = window;
  p.scale2 = scale * 1.44269504088896340736f;
  p.kts = kts;
  p.vts = vts;
  p.y = y;
  p.ldy = ldy;
  p.y_bf16 = y_bf16;
  p.chunk = pl.chunk;
  p.splits = pl.splits;
  p.tile = pl.tile;
  p.slots = rows * H * G;
  p.part_o = static_cast<float*>(ws);
  p.part_ms = reinterpret_cast<float2*>(p.part_o + (size_t)pl.splits * (size_t)p.slots * D);
  if (fmt == FP4Q_NVFP4) {
    if (D == 64) launch<FP4Q_NVFP4, 64>(p, pl, H, B, stream);
    else if (D == 128) launch<FP4Q_NVFP4, 128>(p, pl, H, B, stream);
    else launch<FP4Q_NVFP4, 256>(p, pl, H, B, stream);
  } else {
    if (D == 64) launch<FP4Q_MXFP4, 64>(p, pl, H, B, stream);
    else if (D == 128) launch<FP4Q_MXFP4, 128>(p, pl, H, B, stream);
    else launch<FP4Q_MXFP4, 256>(p, pl, H, B, stream);
  }
}

}  // namespace fp4q
