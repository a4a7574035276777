// attention_tile.hip -- attention over the paged FP4 key/value cache for many
// rows (prompts and chunks of them): the formula of attention.hip, one pass
// over the keys with a running maximum and sum.
//
// What bounds it: the matrix products (4 D operations a row and key) and, on
// the vector units at about the same weight, one exponential a row and key;
// decoding the cache would cost as much again if every wave did it for its
// own rows.  So a workgroup of WAVES waves takes 32 rows a wave (row r of a
// sequence's kv head is query r / G, head r % G of the group) and decodes
// each 64 keys once, into LDS, for all of them: half of its waves decode K,
// half V, so that each SIMD has one of both, from bytes that were loaded two
// steps before; LDS is double-buffered with one barrier a step.
//
// Products are 32x32x16:  S^T = K Q^T  (lane: query lane % 32, and 16 of each
// 32 keys), O^T += V^T P^T, where a lane's own rounded weights are its
// operand: the order of the keys within a product is free, so V stands in
// LDS in the order in which the lanes hold their keys:
//   lane half h, value i of a 32-key tile: key 8 (i / 4) + 4 h + i % 4
// An exponential costs one FMA more, with -m cf as its addend; the rescaling is
// left out while no score passes the maximum by 2^8.
//
// 4 prompts of up to 4096 tokens (32 heads of 128 on 4, 217 GFLOP) take 276 us,
// 787 TFLOP/s; a library product reaches 1225.  A product takes the vector port
// for 12 of its 32 cycles, and the two waves' vector work and products are about
// equal, so at best 2700 cycles of the 4600 that 64 keys take are needed.  Dim 256
// (one wave a SIMD, so that nothing hides its waits): 2 prompts of up to 2048 tokens,
// 16 heads on 4, 35 GFLOP, 164 us; the vector units issue in a third of the cycles.
#include "attention_common.h"

namespace fp4q {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

// Weights are 2^(x cf + nb) up to scores of this many log2 units.  nb is rounded
// anew with each maximum, which weighs older and newer keys apart by up to 2^-16
// of them there (a weight's own rounding: 2^-11 or 2^-8), and by percents at 2^19.
constexpr float FAR = 256.0f;

// Keys of a step.
template <int D> struct TileKeys { static constexpr int N = D <= 128 ? 64 : 32; };

template <int FMT> struct Wide;
template <> struct Wide<FP4Q_NVFP4> {
  static __device__ __forceinline__ v16f mfma(h8 a, h8 b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <> struct Wide<FP4Q_MXFP4> {
  static __device__ __forceinline__ v16f mfma(b8 a, b8 b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

// LDS of one step's keys: K [key][D], V [element][key], both of 2-byte values
// with 16 bytes of padding a row, so that eight neighbouring rows' 16-byte
// reads cover all banks.
template <int D>
struct TileLds {
  static constexpr int TILE_KEYS = TileKeys<D>::N;
  static constexpr int KROW = D * 2 + 16, KBYTES = TILE_KEYS * KROW, KBUFS = 3;
  static constexpr int VROW = TILE_KEYS * 2 + 16, VBYTES = D * VROW;
  static constexpr int V0 = KBUFS * KBYTES;
  static constexpr int BYTES = V0 + 2 * VBYTES;
};

// The cache bytes that a wave decodes for one step: UNITS times 16 keys, which
// stand in one page (its number and address are scalars).  A lane has of K the
// 32-element runs lane, lane + 64, ... of the 16 keys (ITEMS of them), of V four
// tokens' elements lane % 16, lane % 16 + 16, ...
template <int FMT, int D, int TEAM_WAVES>
struct Staged {
  typedef KvLayout<FMT, D> L;
  static constexpr int UNITS = TileKeys<D>::N / 16 / TEAM_WAVES;
  static constexpr int ITEMS = (16 * L::J + 63) / 64;
  static constexpr int VC = D / 32, VS = L::SB;  // dwords of codes and scales of a V unit
  static constexpr int K_W = ITEMS * 5, V_W = VC + VS, W = K_W > V_W ? K_W : V_W;
  uint32_t w[UNITS][W];
  int id[UNITS];    // pages of the step after (-1: none)
  bool good[UNITS]; // are those of the staged step in the cache?
};

// The page table's entries, which no kernel writes while this one runs, through
// the scalar cache.
typedef const __attribute__((address_space(4))) int32_t* TablePtr;

// Asks the scheduler for N products fed by N LDS reads with AHEAD of the reads
// in flight: left alone, it reads, waits and multiplies by turns.
template <int N, int AHEAD>
__device__ __forceinline__ void pipeline_reads() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);  // LDS reads
#pragma unroll
  for (int i = 0; i < N - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, AHEAD, 0);
}

template <int FMT, int D, int WAVES, bool SINK>
__global__ __launch_bounds__(64 * WAVES)
    __attribute__((amdgpu_waves_per_eu(D == 64 ? 4 : D == 128 ? 2 : 1))) void k_attn_tile(AttnArgs p) {
  typedef typename Num<FMT>::vec vec;
  typedef typename Num<FMT>::pair pair;
  typedef KvLayout<FMT, D> L;
  typedef TileLds<D> S;
  constexpr int TILE_KEYS = TileKeys<D>::N, NU = TILE_KEYS / 32;
  constexpr uint32_t ALL_OK = NU == 2 ? 0x01010101u : 0x0101u;
  typedef Staged<FMT, D, WAVES / 2> St;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  // of the last steps, byte u: is the page of keys 16u .. 16u + 15 in the cache?
  // (dim 256 has two units a step: its upper bytes are never written)
  __shared__ uint32_t s_ok[4];

  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go to the XCDs in turn: the (sequence, kv head) is rotated by
  // the row tile, so that a long sequence is not left to a few of them.
  const uint32_t bh = (blockIdx.x + blockIdx.y) % gridDim.x;
  const int b = bh / p.H, h = bh - b * p.H;
  zero_rest<D, 64 * WAVES>(p, b, h);
  // the last rows, which see the most keys, first
  const int n_rows = tile_rows(p, b);
  const int tile_id = min((n_rows + p.tile - 1) / p.tile, (int)gridDim.y) - 1 - (int)blockIdx.y;
  if (tile_id < 0) return;
  const int row0 = tile_id * p.tile;
  const Range rg = tile_range<SINK>(p, b, row0);
  const int split = blockIdx.z;
  if (split >= active_splits(p, rg)) return;
  const int k0 = rg.lo + split * p.chunk;
  const int k1 = split_end(p, rg, k0);
  const int page = 1 << p.page_shift;
  const TablePtr table = (TablePtr)(uintptr_t)(p.table + b * p.ldt);
  const uint32_t n_pages = (uint32_t)min(p.n_pages, (int64_t)0x7FFFFFFF);

  // ---- this wave's rows -----------------------------------------------------
  const int wrow = row0 + wave * 32, row = wrow + col;
  const bool wave_on = wrow < rg.rows;
  const int rr = min(row, rg.rows - 1);
  const int qi = rr / p.G, hh = h * p.G + (rr - qi * p.G);
  const int pos = rg.first + qi;
  const int see_hi = min(rg.hi, pos + 1);
  const int see_lo = first_key(p, pos);
  const int pos_a = rg.first + min(wrow, rg.rows - 1) / p.G;        // the wave's first and
  const int pos_z = rg.first + (min(wrow + 32, rg.rows) - 1) / p.G;  // last position
  float m = -__builtin_inff(), z = 0.0f;
  float lim = m;        // a score above it asks for a new maximum
  float nb = P_BIAS;    // P_BIAS - m cf
  bool far = false;     // is some column's m cf past FAR?
  v16f o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;

  // ---- loading and decoding -------------------------------------------------
  const bool v_team = wave < WAVES / 2;
  const int unit0 = wave % (WAVES / 2);  // its units: unit0, unit0 + WAVES / 2, ...
  St st;
  const int64_t page_stride = (int64_t)p.H * L::bytes(page), head0 = h * (int64_t)L::bytes(page);
  // page numbers of step t
  auto load_ids = [&](int t) {
#pragma unroll
    for (int n = 0; n < St::UNITS; ++n) {
      const int key = k0 + t * TILE_KEYS + 16 * (unit0 + n * (WAVES / 2));
      st.id[n] = key < k1 ? table[real_key<SINK>(p, rg, key) >> p.page_shift] : -1;
    }
  };
  // bytes of step t, from st.id; the K team notes which pages are good
  auto load_bytes = [&](int t) {
#pragma unroll
    for (int n = 0; n < St::UNITS; ++n) {
      const int unit = unit0 + n * (WAVES / 2);
      const bool good = (uint32_t)st.id[n] < n_pages;
      st.good[n] = good;
      // (for a page that is not in the cache some page's bytes, all masked)
      const uint8_t* base = p.cache + (good ? st.id[n] : 0) * page_stride + head0;
      const int slot = real_key<SINK>(p, rg, k0 + t * TILE_KEYS + 16 * unit) & (page - 1);
      if (v_team) {
        uint32_t c[St::VC], s[St::VS];
        load_words(base + L::v_codes(page) + slot * (D / 2) + (uint32_t)(lane * (D / 8)), c);
        load_words(base + L::v_scales(page) + slot * L::SB + (uint32_t)((lane >> 4) * 4 * L::SB), s);
#pragma unroll
        for (int i = 0; i < St::VC; ++i) st.w[n][i] = c[i];
#pragma unroll
        for (int i = 0; i < St::VS; ++i) st.w[n][St::VC + i] = s[i];
      } else {
        const uint8_t *kc = base + slot * (D / 2), *ks = base + L::k_scales(page) + slot * L::SB;
#pragma unroll
        for (int i = 0; i < St::ITEMS; ++i) {
          const uint32_t run = lane + 64 * i;
          if (16 * L::J < 64 && run >= 16 * L::J) continue;
          const w4 u = *reinterpret_cast<const w4*>(kc + run * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) st.w[n][5 * i + e] = u[e];
          if (FMT == FP4Q_NVFP4) st.w[n][5 * i + 4] = *reinterpret_cast<const uint16_t*>(ks + run * 2);
          else st.w[n][5 * i + 4] = ks[run];
        }
        if (lane == 0) reinterpret_cast<uint8_t*>(&s_ok[t & 3])[unit] = good ? 1 : 0;
      }
    }
  };
  // the staged bytes as values in LDS
  uint8_t* const vdst = lds + S::V0 + (lane & 15) * S::VROW + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
  auto decode = [&](int t) {
#pragma unroll
    for (int n = 0; n < St::UNITS; ++n) {
      const int unit = unit0 + n * (WAVES / 2);
      if (v_team) {
        Sub<FMT, D> s;
#pragma unroll
        for (int i = 0; i < St::VC; ++i) s.v[i] = st.w[n][i];
#pragma unroll
        for (int i = 0; i < St::VS; ++i) s.vs[i] = st.w[n][St::VC + i];
        const int key = real_key<SINK>(p, rg, k0 + t * TILE_KEYS + 16 * unit);
        if (!st.good[n] || (key < rg.seen && !(SINK && key + 16 <= p.sinks)) || key + 16 > rg.hi)
          zero_v_scales<FMT, D, SINK>(s, key + 4 * (lane >> 4), !st.good[n], rg.seen, rg.hi, p.sinks);
        uint8_t* dst = vdst + (t & 1) * S::VBYTES + unit * 32;
        v_rows<FMT, D, 0>(s, [&](int run, u32x2 lo, u32x2 hi) {
          *reinterpret_cast<u32x2*>(dst + (32 * run) * S::VROW) = lo;
          *reinterpret_cast<u32x2*>(dst + (32 * run + 16) * S::VROW) = hi;
        });
      } else {
#pragma unroll
        for (int i = 0; i < St::ITEMS; ++i) {
          const int run = lane + 64 * i;
          if (16 * L::J < 64 && run >= 16 * L::J) continue;
          uint8_t* dst = lds + t % S::KBUFS * S::KBYTES + (16 * unit + run / L::J) * S::KROW + run % L::J * 64;
#pragma unroll
          for (int e = 0; e < 4; ++e)  // NVFP4: two blocks in the run
            *reinterpret_cast<vec*>(dst + 16 * e) =
                decode8<FMT>(st.w[n][5 * i + e], k_scale<FMT>(st.w[n][5 * i + 4], e >> 1));
        }
      }
    }
  };

  const int steps = k0 < k1 ? (k1 - k0 + TILE_KEYS - 1) / TILE_KEYS : 0;
  if (steps > 0) {  // on their way while q is loaded
    load_ids(0);
    load_bytes(0);
    load_ids(1);
  }
  vec qf[D / 16];
  float cf;
  {
    const uint16_t* q = p.q + (rg.r0 + qi) * p.ldq + hh * D + half * 8;
    w4 u[D / 16];
#pragma unroll
    for (int st = 0; st < D / 16; ++st) u[st] = *reinterpret_cast<const w4*>(q + 16 * st);
    cf = p.scale2 * (FMT == FP4Q_NVFP4 ? p.kts[h] : 1.0f);
    if constexpr (FMT == FP4Q_MXFP4) {
#pragma unroll
      for (int st = 0; st < D / 16; ++st) qf[st] = __builtin_bit_cast(vec, u[st]);
    } else {
      uint32_t mq = 0;
#pragma unroll
      for (int st = 0; st < D / 16; ++st) mq = max(mq, max_magnitude(u[st]));
      mq = max(mq, (uint32_t)__shfl_xor((int)mq, 32));
      const int sh = q_exponent(mq);
      cf *= __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
      for (int st = 0; st < D / 16; ++st) qf[st] = __builtin_bit_cast(vec, q_to_f16(u[st], sh));
    }
    cf = fmaxf(cf, MIN_FACTOR);
  }

  // ---- the keys ---------------------------------------------------------------
  // One barrier a step.  The V team's waves and the K team's (one of each on a
  // SIMD) go through a step in another order, so that one's products meet the
  // other's vector work:
  //   V team: S of t, V of t + 1 into LDS, weights of t, O += P V of t
  //   K team: K of t + 2 into LDS, weights of t, O += P V of t, S of t + 1
  // In step t K of t and t + 1 and V of t are read, K of t + 2 and V of t + 1
  // written: three K buffers and two V buffers do.  Of the page flags, that of t
  // is read and that of t + 3 written (with the load): four do.
  // this wave's steps (those that some row of it sees)
  // (a window that skip is taken from begins after it, and so do the rows' positions)
  const int last_kt = pos_z - rg.skip;
  int t_on = 0, t_off = wave_on ? min(steps, last_kt < k0 ? 0 : (last_kt - k0) / TILE_KEYS + 1) : 0;
  if (p.window > 0) t_on = max(0, first_key(p, pos_a) - rg.skip - k0) / TILE_KEYS;
  const int t_sink = SINK ? max(0, p.sink_end - k0) / TILE_KEYS : 0;  // steps of the first tokens
  auto is_on = [&](int t) { return (t >= t_on || (SINK && t < t_sink)) && t < t_off; };
  v16f x[NU];
  vec pb[2 * NU];
  const uint8_t* const kb = lds + col * S::KROW + half * 16;
  const uint8_t* const vb = lds + S::V0 + col * S::VROW + half * 16;
  auto score = [&](int t) {  // S of step t
    const uint8_t* k = kb + t % S::KBUFS * S::KBYTES;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) x[u][r] = 0.0f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
      for (int u = 0; u < NU; ++u)
        x[u] = Wide<FMT>::mfma(*reinterpret_cast<const vec*>(k + u * 32 * S::KROW + s * 32), qf[s], x[u]);
    pipeline_reads<NU * D / 16, D == 64 ? 2 : 8>();
  };
  if (steps > 0) {
    decode(0);
    load_bytes(1);
    load_ids(2);
    if (!v_team) {
      decode(1);
      load_bytes(2);
      load_ids(3);
    }
    __syncthreads();
    if (!v_team && is_on(0)) score(0);
  }
  for (int t = 0; t < steps; ++t) {
    const bool on = is_on(t);
    if (v_team && on) score(t);
    const int ahead = v_team ? t + 1 : t + 2;
    decode(ahead);
    load_bytes(ahead + 1);
    load_ids(ahead + 2);
    if (on) {
      const uint32_t ok = s_ok[t & 3];
      const int kt = real_key<SINK>(p, rg, k0 + t * TILE_KEYS);
      const bool whole = (__builtin_amdgcn_readfirstlane(ok) & ALL_OK) == ALL_OK && kt + TILE_KEYS <= pos_a + 1 &&
                         kt + TILE_KEYS <= rg.hi &&
                         (kt >= first_key(p, pos_z) || (SINK && kt + TILE_KEYS <= p.sinks));
      if (!whole) {
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int key = kt + 32 * u + 8 * (r >> 2) + 4 * half + (r & 3);
            if (!((ok >> (8 * (2 * u + (r >> 3)))) & 1) || (key < see_lo && !(SINK && key < p.sinks)) ||
                key >= see_hi)
              x[u][r] = -__builtin_inff();
          }
      }
      float top = x[0][0];
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, x[u][r]);
      top = other_half_max(top);
      if (__any(top > lim)) {
        // (columns whose maximum stays keep it)
        const float mt = top > lim ? top : m;
        const float f = m > -__builtin_inff() ? __builtin_amdgcn_exp2f((m - mt) * cf) : 0.0f;
        m = mt;
        if (m > -__builtin_inff()) {
          lim = m + P_SLACK / cf;
          nb = __builtin_fmaf(-m, cf, P_BIAS);
        }
        far = __any(fabsf(m * cf) > FAR && m > -__builtin_inff());
        z *= f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[i][r] *= f;
      }
      // 2^(x cf + nb), nb = P_BIAS - m cf rounded (past FAR the difference is taken
      // first).
      float add = nb;
      if (far) {
        const float base = m > -__builtin_inff() ? m : 0.0f;
        add = P_BIAS;
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r) x[u][r] -= base;
      }
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w4 pk;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            v2f v;
            v[0] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][8 * e + 2 * r], cf, add));
            v[1] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][8 * e + 2 * r + 1], cf, add));
            z += v[0] + v[1];
            pk[r] = as_u32(__builtin_convertvector(v, pair));
          }
          pb[2 * u + e] = __builtin_bit_cast(vec, pk);
        }
      const uint8_t* v = vb + (t & 1) * S::VBYTES;
#pragma unroll
      for (int e = 0; e < 2 * NU; ++e)
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          o[i] = Wide<FMT>::mfma(*reinterpret_cast<const vec*>(v + i * 32 * S::VROW + e * 32), pb[e], o[i]);
      pipeline_reads<NU * D / 16, D == 64 ? 2 : 8>();
    }
    if (!v_team && is_on(t + 1)) score(t + 1);
    __syncthreads();
  }

  // ---- the results ------------------------------------------------------------
  z += __shfl_xor(z, 32);
  if (row >= rg.rows) return;
  if (p.splits == 1) {
    const float f = z > 0.0f ? (FMT == FP4Q_NVFP4 ? p.vts[h] : 1.0f) / z : 0.0f;
    const int64_t at = (rg.r0 + qi) * p.ldy + hh * D + 4 * half;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v4f t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = o[i][4 * r + e] * f;
        store_out(p, at + 32 * i + 8 * r, t);
      }
  } else {
    const int64_t s = split * p.slots + (rg.r0 + qi) * (int64_t)(p.H * p.G) + hh;
    float f;
    const float whole = whole_max(m, cf, f);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v4f t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = o[i][4 * r + e] * f;
        *reinterpret_cast<v4f*>(p.part_o + s * D + 32 * i + 8 * r + 4 * half) = t;
      }
    if (half == 0) p.part_ms[s] = make_float2(whole, z * f);
  }
}

template <int FMT, int D, int WAVES>
void launch(const AttnArgs& p, int tiles, int B, hipStream_t stream) {
  const dim3 grid((unsigned)(B * p.H), (unsigned)tiles, (unsigned)p.splits);
  if (p.sink_end > 0)
    hipLaunchKernelGGL((k_attn_tile<FMT, D, WAVES, true>), grid, dim3(64 * WAVES), TileLds<D>::BYTES,
                       stream, p);
  else
    hipLaunchKernelGGL((k_attn_tile<FMT, D, WAVES, false>), grid, dim3(64 * WAVES), TileLds<D>::BYTES,
                       stream, p);
}

template <int FMT>
void launch_dim(int D, const AttnArgs& p, int tiles, int B, hipStream_t stream) {
  if (D == 64) {
    if (p.tile == 256) launch<FMT, 64, 8>(p, tiles, B, stream);
    else launch<FMT, 64, 4>(p, tiles, B, stream);
  } else if (D == 128) {
    if (p.tile == 256) launch<FMT, 128, 8>(p, tiles, B, stream);
    else launch<FMT, 128, 4>(p, tiles, B, stream);
  } else {
    launch<FMT, 256, 4>(p, tiles, B, stream);
  }
}

}  // namespace

void launch_attention_tile(int fmt, int D, const AttnArgs& p, int tiles, int B, hipStream_t stream) {
  if (fmt == FP4Q_NVFP4) launch_dim<FP4Q_NVFP4>(D, p, tiles, B, stream);
  else launch_dim<FP4Q_MXFP4>(D, p, tiles, B, stream);
}

}  // namespace fp4q
