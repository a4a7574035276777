// attention.hip -- attention over the paged FP4 key/value cache (defined in
// include/fp4q.h): per new token i and head,
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i.k_j - m_i),
// over the keys j of its sequence with j <= position(i) (and j > position(i)
// - window, or j among the first tokens that stay visible), in one pass over the keys with a running maximum and sum.
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
//
// Few rows (this file): 64 x 1 token over up to 8192 keys (249 MB) take 70-72 us,
// 3.5 TB/s where a copy reaches 4.8, and the join of the splits 7.  The vector units
// issue (decoding, for the most part) in 52% of the cycles, the waves wait for the
// cache's bytes in 47% of theirs.  One token over 777 keys is one wave's chain of
// four steps: 10.6 us.  Many rows: attention_tile.hip.
#include "attention_common.h"

namespace fp4q {

namespace {

// WAVES waves share the keys of a (sequence, kv head, rows, split): wave w
// takes steps w, w + WAVES, ...  With few rows the cache's bytes bound it: K of
// the next step is loaded as soon as this step's is used up, into the same
// registers (few enough for three waves on a SIMD), then V, and the numbers of
// their pages one step before that.
template <int FMT, int D, int NC, int WAVES, bool SINK>
__global__ __launch_bounds__(64 * WAVES, D == 64 ? 4 : D == 128 && NC == 1 && WAVES == 4 ? 3 : 2) void k_attn_split(AttnArgs p) {
  typedef typename Num<FMT>::vec vec;
  typedef typename Num<FMT>::pair pair;
  typedef KvLayout<FMT, D> L;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go to the XCDs in turn: the (sequence, kv head) runs fastest,
  // rotated by the split, so that no XCD has all of the long sequences' last splits.
  const uint32_t bh = (blockIdx.x + blockIdx.z) % gridDim.x;
  const int b = bh / p.H, h = bh - b * p.H, row0 = blockIdx.y * p.tile;
  if (row0 >= tile_rows(p, b)) {
    zero_rest<D, 64 * WAVES>(p, b, h);
    return;
  }
  const Range rg = tile_range<SINK>(p, b, row0);
  const int split = blockIdx.z;
  if (split >= active_splits(p, rg)) return;
  const int k0 = rg.lo + split * p.chunk;
  const int k1 = split_end(p, rg, k0);

  const int page = 1 << p.page_shift;
  const int32_t* table = p.table + b * p.ldt;
  const uint32_t n_pages = (uint32_t)min(p.n_pages, (int64_t)0x7FFFFFFF);
  const int64_t page_stride = (int64_t)p.H * L::bytes(page);
  const uint8_t* const head = p.cache + h * (int64_t)L::bytes(page);
  Sub<FMT, D> st[2];             // the step's two subtiles
  Buffer buf[2];                 // the pages of the step after
  bool good[2], next_good[2];    // is the step's page in the cache?
  int ids[2];                    // page numbers of the step after that
  auto load_ids = [&](int kt) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      ids[u] = table[real_key<SINK>(p, rg, min(kt + 16 * u + (lane & 1), k1 - 1)) >> p.page_shift];
  };
  auto next_k = [&](int kt) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int id = __builtin_amdgcn_readfirstlane(ids[u]), key = kt + 16 * u;
      next_good[u] = (uint32_t)id < n_pages && key < k1;
      // (for a page that is not in the cache some page's bytes, all masked)
      buf[u] = page_buffer(head + (next_good[u] ? id : 0) * page_stride, L::bytes(page));
      load_k<FMT, D>(buf[u], page, real_key<SINK>(p, rg, key) & (page - 1), lane, st[u]);
    }
  };
  auto next_v = [&](int kt) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      load_v<FMT, D>(buf[u], page, real_key<SINK>(p, rg, kt + 16 * u) & (page - 1), lane, st[u]);
  };
  constexpr int STRIDE = WAVES * KEYS;
  int kt = k0 + wave * KEYS;
  if (kt < k1) {
    load_ids(kt);
    next_k(kt);
    next_v(kt);
    load_ids(kt + STRIDE);
  }

  vec qf[NC][D / 32];
  float cf[NC], m[NC], z[NC];
  int see_lo[NC], see_hi[NC];  // keys the column sees: [see_lo, see_hi), and the first ones
  v4f o[NC][D / 16];
  const float c0 = p.scale2 * (FMT == FP4Q_NVFP4 ? p.kts[h] : 1.0f);
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int rr = min(row0 + n * ROWS + c, rg.rows - 1);
    const int qi = rr / p.G, hh = h * p.G + (rr - qi * p.G);
    load_q<FMT, D>(p.q + (rg.r0 + qi) * p.ldq + hh * D, g, c0, qf[n], cf[n]);
    see_hi[n] = min(rg.hi, rg.first + qi + 1);
    see_lo[n] = first_key(p, rg.first + qi);
    m[n] = -__builtin_inff();
    z[n] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[n][i] = {0.0f, 0.0f, 0.0f, 0.0f};
  }
  // a step inside [all_lo, all_hi) needs no mask
  const int last = min(rg.rows, row0 + p.tile) - 1;
  const int all_hi = min(rg.hi, rg.first + row0 / p.G + 1);
  const int all_lo = first_key(p, rg.first + last / p.G);

  for (; kt < k1; kt += STRIDE) {
    good[0] = next_good[0];
    good[1] = next_good[1];
    v4f x[NC][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int n = 0; n < NC; ++n) x[n][u] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const vec a = decode_k<FMT, D>(st[u], i);
#pragma unroll
        for (int n = 0; n < NC; ++n) x[n][u] = Num<FMT>::mfma(a, qf[n][i], x[n][u]);
        __builtin_amdgcn_sched_barrier(0);  // (decoding ahead would cost registers, and so waves)
      }
    }
    next_k(kt + STRIDE);  // (past the last step: some page's bytes, not used)
    const int key0 = real_key<SINK>(p, rg, kt);
    const bool whole = good[0] && good[1] && (key0 >= all_lo || (SINK && key0 + KEYS <= p.sinks)) &&
                       key0 + KEYS <= all_hi;
    float mt[NC], up = 0.0f;  // does some column's maximum run ahead of its kept one?
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = key0 + 16 * u + 4 * g + r;
            if (!good[u] || (key < see_lo[n] && !(SINK && key < p.sinks)) || key >= see_hi[n])
              x[n][u][r] = -__builtin_inff();
          }
      }
      const float t = fmaxf(fmaxf(fmaxf(x[n][0][0], x[n][0][1]), fmaxf(x[n][0][2], x[n][0][3])),
                            fmaxf(fmaxf(x[n][1][0], x[n][1][1]), fmaxf(x[n][1][2], x[n][1][3])));
      mt[n] = fmaxf(other_half_max(other_quarter_max(t)), m[n]);
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
    vec pb[NC];
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
    if (!whole) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        zero_v_scales<FMT, D, SINK>(st[u], key0 + 16 * u + 4 * g, !good[u], rg.seen, rg.hi, p.sinks);
    }
    pv_all<FMT, D, 0, NC>(st[0], st[1], pb, o);
    next_v(kt + STRIDE);
    load_ids(kt + 2 * STRIDE);
  }

  // The waves' results meet: common maximum, summed sums, and the outputs added
  // pairwise, the upper half of the waves to the lower one.
  __shared__ float s_m[WAVES][NC * ROWS], s_z[WAVES][NC * ROWS];
  __shared__ v4f s_o[WAVES / 2][D / 16][64];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    z[n] += __shfl_xor(z[n], 16);
    z[n] += __shfl_xor(z[n], 32);
    if (g == 0) {
      s_m[wave][n * ROWS + c] = m[n];  // (m c, rounded, would weigh the waves apart)
      s_z[wave][n * ROWS + c] = z[n];
    }
  }
  __syncthreads();
  const float vt = FMT == FP4Q_NVFP4 ? p.vts[h] : 1.0f;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    float mm = -__builtin_inff(), zz = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) mm = fmaxf(mm, s_m[w][n * ROWS + c]);
    const float base = mm > -__builtin_inff() ? mm : 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
      zz += s_z[w][n * ROWS + c] * __builtin_amdgcn_exp2f((s_m[w][n * ROWS + c] - base) * cf[n]);
    const float mine = __builtin_amdgcn_exp2f((m[n] - base) * cf[n]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[n][i][r] *= mine;
#pragma unroll
    for (int half = WAVES / 2; half > 0; half >>= 1) {
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) s_o[wave - half][i][lane] = o[n][i];
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const v4f t = s_o[wave][i][lane];
#pragma unroll
          for (int r = 0; r < 4; ++r) o[n][i][r] += t[r];
        }
      }
      __syncthreads();
    }
    const int row = row0 + n * ROWS + c;
    if (wave > 0 || row >= rg.rows) continue;
    const int qi = row / p.G, hh = h * p.G + (row - qi * p.G);
    if (p.splits == 1) {
      const float f = zz > 0.0f ? vt / zz : 0.0f;
      const int64_t at = (rg.r0 + qi) * p.ldy + hh * D + 4 * g;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        v4f t;
#pragma unroll
        for (int r = 0; r < 4; ++r) t[r] = o[n][i][r] * f;
        store_out(p, at + 16 * i, t);
      }
    } else {
      const int64_t s = split * p.slots + (rg.r0 + qi) * (int64_t)(p.H * p.G) + hh;
      float f;
      const float whole = whole_max(mm, cf[n], f);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        v4f t;
#pragma unroll
        for (int r = 0; r < 4; ++r) t[r] = o[n][i][r] * f;
        *reinterpret_cast<v4f*>(p.part_o + s * D + 16 * i + 4 * g) = t;
      }
      if (g == 0) p.part_ms[s] = make_float2(whole, zz * f);
    }
  }
  zero_rest<D, 64 * WAVES>(p, b, h);
}

// Joins the splits of a row: p.join groups of D / 4 lanes for each (new token,
// head), each over every p.join-th split with a running maximum, joined in LDS.
template <int FMT, int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs p) {
  constexpr int LANES = D / 4;
  __shared__ v4f s_o[256];
  __shared__ float2 s_ms[256];
  const int t = threadIdx.x, d = t % LANES;
  const int grp = t / LANES % p.join;
  const int64_t s = (int64_t)blockIdx.x * (256 / LANES / p.join) + t / (LANES * p.join);
  const int heads = p.H * p.G;
  const int64_t row = s / heads;
  const int hh = (int)(s - row * heads);
  int n = 0;
  if (s < p.slots && row >= p.off[0] && row < p.off[p.B]) {
    const int b = kv_sequence(p.off, p.B, row);
    const int qi = (int)(row - p.off[b]), tile = (qi * p.G + hh % p.G) / p.tile;
    if (qi < p.max_new) n = min(active_splits(p, p.sink_end > 0 ? tile_range<true>(p, b, tile * p.tile)
                                                          : tile_range<false>(p, b, tile * p.tile)),
                              p.splits);
  }
  float m = -__builtin_inff(), z = 0.0f;
  v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = grp; i < n; i += p.join) {
    const float2 ms = p.part_ms[i * p.slots + s];
    const v4f a = *reinterpret_cast<const v4f*>(p.part_o + (i * p.slots + s) * D + 4 * d);
    const float mn = fmaxf(m, ms.x), base = mn > -__builtin_inff() ? mn : 0.0f;
    const float f = __builtin_amdgcn_exp2f(m - base), fa = __builtin_amdgcn_exp2f(ms.x - base);
    m = mn;
    z = z * f + ms.y * fa;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(a[r], fa, o[r] * f);
  }
  if (p.join > 1) {
    s_o[t] = o;
    s_ms[t] = make_float2(m, z);
    __syncthreads();
    if (grp > 0) return;
    for (int i = 1; i < p.join; ++i) {
      const float2 ms = s_ms[t + i * LANES];
      const v4f a = s_o[t + i * LANES];
      const float mn = fmaxf(m, ms.x), base = mn > -__builtin_inff() ? mn : 0.0f;
      const float f = __builtin_amdgcn_exp2f(m - base), fa = __builtin_amdgcn_exp2f(ms.x - base);
      m = mn;
      z = z * f + ms.y * fa;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(a[r], fa, o[r] * f);
    }
  }
  if (s >= p.slots) return;
  // (n = 0: a row past the last sequence's or past max_new gives 0)
  const float f = z > 0.0f ? (FMT == FP4Q_NVFP4 ? p.vts[hh / p.G] : 1.0f) / z : 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] *= f;
  store_out(p, row * p.ldy + hh * D + 4 * d, o);
}

// How a call is split: a function of host numbers only, so that the workspace
// query and the launch agree.  Its rules, with what the other choice takes (us a
// call; NVFP4, 8 heads of 128 on a kv head where nothing else is said):
//   wide    more than 32 rows a kv head.  8 x 8 kv heads over 4096 keys: 24 rows 30.6,
//           wide 46.5; 48 rows 49.6 either way; 64 rows 52.0, not wide 56.5 (dim 64: 35.8
//           and 31.4, dim 256: 107 and 110, at 48 rows 103 and 82)
//   nc      17 to 32 rows in one pass: 30.6, in two 31.7 (dim 64 21.2 and 22.8)
//   tile    256 rows from 129 on: 160 rows 60.5, by 128 84.0; 1024 rows 182 and 262
//   waves   eight with at most 256 (sequence, kv head)s and 2048 keys.  256 of them: 777
//           keys 11.6, split over workgroups of four 18.2; 2048 keys 19.2 and 30.4.  The
//           rule is too wide for few of them (8: 777 keys 10.7 and 9.9, 2048 keys 17.5 and
//           10.4) and too narrow above (512, 777 keys: 28.3 by four, 21.7 by eight)
//   want    workgroups asked for.  64 sequences of up to 8192 keys: 84, 80, 77.5, 90 for 1024,
//           2048, 4096, 8192; 3 of up to 131072: 63, 58, 57, 67; of equal lengths 2048 would do
//           (64 x 8192: 127, with 4096 142).  wide: 512 + 83 tokens in a window of 4096 keys,
//           dim 64: 64, 53, 64 for 256, 512, 1024; equal lengths 88 for 256 and 104 for 512
//   least   keys of a split.  8 (sequence, kv head)s over 16384 keys: 18.2, 14.0, 13.1, 16.1 for
//           128, 256, 512, 1024; over 4096: 10.0, 10.5, 12.1, 15.4.  wide: 64 tokens over 65536
//           keys 53.5, 38.8, 47.3 for 256, 512, 1024
//   sinks   a window with first tokens: most sequences are longer than it and see equally
//           many keys, so few rows take as many workgroups as run at once (one split from
//           there on), wide ones 256.  64 sequences of 8 kv heads over 4096 + 4 keys: 72 us
//           in one split, by want and least 93; 8, 32, 48 of them 20, 40, 54 and 23, 62, 79;
//           dim 256 70 and 120; 1024 tokens of one sequence 163, for 512 workgroups 192.
//           Sequences that are shorter than the window lose: 32 of 256 to 4096 keys in a
//           window of 4000 35, for twice the workgroups 28.  Eight waves from 64 (sequence,
//           kv head)s on: 8 of them over 1028 keys 11.8, by eight 12.4
//           Wide: 128 rows where 256 would leave half of the CUs without work (605 tokens of
//           2 kv heads in a window of 31 18.8, by 256 23.1), and 256 keys a split from 1024
//           keys on (40 tokens over 3000 keys 23, by 512 30; 377 keys 25.8 and 28.3)
//   join    lane groups on a row's splits, four to eight splits each.  171 splits: 121 by one
//           group, 115.5 by this rule and by half as many
struct Plan {
  bool wide;  // many rows: k_attn_tile
  int nc, waves, tile, step, chunk, splits, join;
  int64_t tiles;
};

Plan attn_plan(int D, int B, int H, int G, int64_t max_new, int64_t max_len, int window, int sinks) {
  Plan p;
  const int64_t rows = max_new * G;
  const bool sink = sinks > 0 && window > 0;
  p.wide = rows > 2 * ROWS;
  p.nc = rows > ROWS && D <= 128 ? 2 : 1;
  p.tile = p.wide ? (rows > 128 && D <= 128 ? 256 : 128) : ROWS * p.nc;
  if (sink && p.tile == 256 && (rows + 255) / 256 <= 128 / (B * (int64_t)H)) p.tile = 128;
  p.step = p.wide ? 64 : KEYS;
  p.tiles = (rows + p.tile - 1) / p.tile;
  int64_t keys = max_len;
  if (window > 0) {
    int64_t seen = (int64_t)window + (p.wide ? (p.tile + G - 1) / G + 1 : max_new) + p.step;
    if (sinks > 0) seen += ((int64_t)sinks + p.step - 1) / p.step * p.step;
    keys = keys < seen ? keys : seen;
  }
  int64_t groups = B * (int64_t)H * p.tiles;
  if (groups > (1 << 30)) groups = 1 << 30;  // (keys * groups stays below 2^63)
  // eight waves on the keys of each (sequence, kv head), none to join
  p.waves = !p.wide && groups <= 256 && keys <= 2048 && p.nc == 1 && D <= 128 ? 8 : 4;
  const int64_t want = p.wide ? (sink ? 256 : 512) : 4096;
  int64_t chunk = (keys * groups + want - 1) / want;
  const int64_t least = p.wide ? (sink && keys >= 1024 ? 256 : 512) : p.waves == 8 ? 2048 : 256;
  chunk = chunk < least ? least : chunk;
  chunk = (chunk + p.step - 1) / p.step * p.step;
  p.chunk = (int)(chunk < (1 << 30) ? chunk : (1 << 30));
  if (sink && !p.wide) {
    p.waves = groups > 64 && groups <= 256 && keys <= 2048 && p.nc == 1 && D <= 128 ? 8 : 4;
    const int64_t at_once = 256 * (D == 64 ? 4 : D == 128 && p.nc == 1 ? 3 : 2);
    int64_t n = p.waves == 8 ? 1 : at_once / groups;
    n = n < keys / 256 ? n : keys / 256;
    n = n > 1 ? n : 1;
    chunk = ((keys + n - 1) / n + p.step - 1) / p.step * p.step;
    chunk = chunk > p.step ? chunk : p.step;  // (max_len may be 0)
    p.chunk = (int)(chunk < (1 << 30) ? chunk : (1 << 30));
  }
  p.splits = (int)((keys + p.chunk - 1) / p.chunk);
  if (p.splits < 1) p.splits = 1;
  p.join = 1;
  while (p.join * 4 < p.splits && p.join < 1024 / D) p.join *= 2;
  return p;
}

template <int FMT, int D, bool SINK>
void launch_split(const AttnArgs& p, const Plan& pl, int H, int B, hipStream_t stream) {
  const dim3 grid((unsigned)(B * H), (unsigned)pl.tiles, (unsigned)pl.splits), thr(64 * pl.waves);
  if constexpr (D <= 128) {
    if (pl.nc == 2) hipLaunchKernelGGL((k_attn_split<FMT, D, 2, 4, SINK>), grid, thr, 0, stream, p);
    else if (pl.waves == 4) hipLaunchKernelGGL((k_attn_split<FMT, D, 1, 4, SINK>), grid, thr, 0, stream, p);
    else hipLaunchKernelGGL((k_attn_split<FMT, D, 1, 8, SINK>), grid, thr, 0, stream, p);
  } else {
    hipLaunchKernelGGL((k_attn_split<FMT, D, 1, 4, SINK>), grid, thr, 0, stream, p);
  }
}

template <int FMT, int D>
void launch(const AttnArgs& p, const Plan& pl, int H, int B, hipStream_t stream) {
  if (pl.wide) launch_attention_tile(FMT, D, p, (int)pl.tiles, B, stream);
  else if (p.sink_end > 0) launch_split<FMT, D, true>(p, pl, H, B, stream);
  else launch_split<FMT, D, false>(p, pl, H, B, stream);
  if (pl.splits > 1) {
    const int per = 1024 / D / pl.join;  // rows and heads of a workgroup
    hipLaunchKernelGGL((k_attn_join<FMT, D>), dim3((unsigned)((p.slots + per - 1) / per)), dim3(256),
                       0, stream, p);
  }
}

}  // namespace

// Sizes that the launch can hold.
bool attention_shape_ok(int64_t rows, int D, int B, int H, int G, int64_t max_new, int64_t max_len,
                        int window, int sinks) {
  const int64_t heads = (int64_t)H * G, most = (int64_t)1 << 31;
  if (G > 128 || B > 65535 || (int64_t)B * H >= (1 << 22) || rows >= most / heads ||
      max_new >= most / heads || max_len >= most)
    return false;
  const Plan pl = attn_plan(D, B, H, G, max_new, max_len, window, sinks);
  return pl.tiles <= 65535 && pl.splits <= 65535;  // (the grid's second and third dimension)
}

size_t attention_workspace_bytes(int64_t rows, int D, int B, int H, int G, int64_t max_new,
                                 int64_t max_len, int window, int sinks) {
  const Plan pl = attn_plan(D, B, H, G, max_new, max_len, window, sinks);
  return pl.splits > 1 ? (size_t)pl.splits * (size_t)(rows * H * G) * (size_t)(D + 2) * 4 : 0;
}

void launch_attention(int fmt, const uint8_t* cache, int64_t n_pages, int page_shift, int H, int D,
                      const int32_t* off, int B, const int32_t* table, int64_t ldt, int64_t table_cols,
                      const int32_t* lens, const uint16_t* q, int64_t ldq, int64_t rows, int G,
                      int64_t max_new, int64_t max_len, int window, int sinks, float scale, const float* kts,
                      const float* vts, void* y, int y_bf16, int64_t ldy, void* ws,
                      hipStream_t stream) {
  const Plan pl = attn_plan(D, B, H, G, max_new, max_len, window, sinks);
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
  const int64_t held = table_cols << page_shift;
  p.cap = (int)(held < max_len ? held : max_len);
  p.lens = lens;
  p.q = q;
  p.ldq = ldq;
  p.rows = (int)rows;
  p.max_new = (int)max_new;
  p.window = window;
  // (without a window every key stays visible)
  p.sinks = window > 0 ? (sinks < p.cap ? sinks : p.cap) : 0;
  p.sink_end = (p.sinks + pl.step - 1) & ~(pl.step - 1);
  p.scale2 = scale * 1.44269504088896340736f;
  p.kts = kts;
  p.vts = vts;
  p.y = y;
  p.ldy = ldy;
  p.y_bf16 = y_bf16;
  p.chunk = pl.chunk;
  p.splits = pl.splits;
  p.tile = pl.tile;
  p.step = pl.step;
  p.join = pl.join;
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
