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
#include "attention_common.h"

namespace fp4q {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int TILE_KEYS = 64;

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
  static constexpr int KROW = D * 2 + 16;
  static constexpr int VROW = TILE_KEYS * 2 + 16;
  static constexpr int V0 = TILE_KEYS * KROW;
  static constexpr int BYTES = V0 + D * VROW;
};

// The cache bytes that a thread decodes for one step.  K: 32 elements of one
// key; V: the four tokens of a group, elements c, c + 16, ...
template <int FMT, int D, int TEAM>
struct Staged {
  typedef KvLayout<FMT, D> L;
  static constexpr int K_ITEMS = TILE_KEYS * (D / 32);
  static constexpr int V_ITEMS = TILE_KEYS * 4;
  static constexpr int NK = (K_ITEMS + TEAM - 1) / TEAM;
  static constexpr int NV = (V_ITEMS + TEAM - 1) / TEAM;
  static constexpr int VC = D / 32, VS = L::SB;  // dwords of codes and scales of a V item
  static constexpr int NK_W = NK * 5, NV_W = NV * (VC + VS);
  uint32_t w[NK_W > NV_W ? NK_W : NV_W];
  int id[NK > NV ? NK : NV];  // pages of the step after
};

__device__ __forceinline__ float other_half_max(float v) {
  const u32x2 r = __builtin_bit_cast(
      u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

template <int FMT, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D <= 128 ? 2 : 1) void k_attn_tile(AttnArgs p) {
  typedef typename Num<FMT>::vec vec;
  typedef typename Num<FMT>::pair pair;
  typedef KvLayout<FMT, D> L;
  typedef TileLds<D> S;
  constexpr int TEAM = 32 * WAVES;  // threads that decode K; as many decode V
  typedef Staged<FMT, D, TEAM> St;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // two steps' K and V
  // of the last steps, byte u: is the page of keys 16u .. 16u + 15 in the cache?
  __shared__ uint32_t s_ok[4];

  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go to the XCDs in turn: the (sequence, kv head) is rotated by
  // the row tile, so that a long sequence is not left to a few of them.
  const uint32_t bh = (blockIdx.x + blockIdx.y) % gridDim.x;
  const int b = bh / p.H, h = bh - b * p.H;
  // the last rows, which see the most keys, first
  const int row0 = (int)(gridDim.y - 1 - blockIdx.y) * p.tile;
  const int n_rows = (p.off[b + 1] - p.off[b]) * p.G;
  if (row0 >= n_rows) return;
  const Range rg = tile_range(p, b, row0);
  const int split = blockIdx.z;
  if (split >= active_splits(p, rg)) return;
  const int k0 = rg.lo + split * p.chunk;
  const int k1 = min(rg.hi, k0 + p.chunk);
  const int page = 1 << p.page_shift;
  const int32_t* table = p.table + b * p.ldt;
  const uint32_t n_pages = (uint32_t)min(p.n_pages, (int64_t)0x7FFFFFFF);

  // ---- this wave's rows -----------------------------------------------------
  const int wrow = row0 + wave * 32, row = wrow + col;
  const bool wave_on = wrow < rg.rows;
  const int rr = min(row, rg.rows - 1);
  const int qi = rr / p.G, hh = h * p.G + (rr - qi * p.G);
  const int pos = rg.first + qi;
  const int see_hi = min(rg.hi, pos + 1);
  const int see_lo = p.window > 0 ? pos - p.window + 1 : 0;
  const int pos_a = rg.first + min(wrow, rg.rows - 1) / p.G;        // the wave's first and
  const int pos_z = rg.first + (min(wrow + 32, rg.rows) - 1) / p.G;  // last position
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
    cf = fmaxf(cf, 1e-37f);
  }
  float m = -__builtin_inff(), z = 0.0f;
  float lim = m;        // a score above it asks for a new maximum
  float nb = P_BIAS;    // P_BIAS - m cf
  bool far = false;     // is some column's m cf so large that nb loses its fraction?
  v16f o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;

  // ---- loading and decoding -------------------------------------------------
  const bool v_team = wave < WAVES / 2;
  const int tid = threadIdx.x & (TEAM - 1);
  St st;
  // page numbers of the step that starts at kt (past the last key: any)
  auto load_ids = [&](int kt) {
    if (v_team) {
#pragma unroll
      for (int n = 0; n < St::NV; ++n)
        st.id[n] = table[min(kt + 4 * ((tid + n * TEAM) >> 4), k1 - 1) >> p.page_shift];
    } else {
#pragma unroll
      for (int n = 0; n < St::NK; ++n)
        st.id[n] = table[min(kt + (tid + n * TEAM) / (D / 32), k1 - 1) >> p.page_shift];
    }
  };
  // bytes of the step at kt, from st.id; the K team notes which pages are good
  auto load_bytes = [&](int kt) {
    if (v_team) {
#pragma unroll
      for (int n = 0; n < St::NV; ++n) {
        const int item = tid + n * TEAM, key = kt + 4 * (item >> 4);
        const bool good = (uint32_t)st.id[n] < n_pages;
        const int64_t id = good ? st.id[n] : 0;  // (some page's bytes: their scales become 0)
        const uint8_t* base = p.cache + (id * p.H + h) * (int64_t)L::bytes(page);
        const int slot = key & (page - 1);
        uint32_t* w = st.w + n * (St::VC + St::VS);
        uint32_t c[St::VC], s[St::VS];
        load_words(base + L::v_codes(page) + slot * (D / 2) + (item & 15) * (D / 8), c);
        load_words(base + L::v_scales(page) + slot * L::SB, s);
#pragma unroll
        for (int i = 0; i < St::VC; ++i) w[i] = c[i];
#pragma unroll
        for (int i = 0; i < St::VS; ++i) w[St::VC + i] = s[i];
      }
    } else {
#pragma unroll
      for (int n = 0; n < St::NK; ++n) {
        const int item = tid + n * TEAM, key = kt + item / (D / 32), part = item % (D / 32);
        if (St::K_ITEMS % TEAM != 0 && item >= St::K_ITEMS) continue;
        const bool good = (uint32_t)st.id[n] < n_pages;
        const int64_t id = good ? st.id[n] : 0;
        const uint8_t* base = p.cache + (id * p.H + h) * (int64_t)L::bytes(page);
        const int slot = key & (page - 1);
        const w4 u = *reinterpret_cast<const w4*>(base + slot * (D / 2) + part * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) st.w[n * 5 + i] = u[i];
        const uint8_t* ks = base + L::k_scales(page) + slot * L::SB;
        if (FMT == FP4Q_NVFP4) st.w[n * 5 + 4] = reinterpret_cast<const uint16_t*>(ks)[part];
        else st.w[n * 5 + 4] = ks[part];
        if (part == 0 && (key & 15) == 0)
          reinterpret_cast<uint8_t*>(&s_ok[(key / TILE_KEYS) & 3])[(key >> 4) & 3] = good ? 1 : 0;
      }
    }
  };
  // the staged bytes as values in LDS
  auto decode = [&](int kt, int buf, uint32_t bad) {
    uint8_t* base = lds + buf * S::BYTES;
    if (v_team) {
#pragma unroll
      for (int n = 0; n < St::NV; ++n) {
        const int item = tid + n * TEAM, grp = item >> 4, c = item & 15;
        Sub<FMT, D> s;
        uint32_t* w = st.w + n * (St::VC + St::VS);
#pragma unroll
        for (int i = 0; i < St::VC; ++i) s.v[i] = w[i];
#pragma unroll
        for (int i = 0; i < St::VS; ++i) s.vs[i] = w[St::VC + i];
        const int key = kt + 4 * grp;
        if (((bad >> n) & 1) || key < rg.seen || key + 4 > rg.hi)
          zero_v_scales<FMT, D>(s, key, (bad >> n) & 1, rg.seen, rg.hi);
        uint8_t* dst = base + S::V0 + c * S::VROW + (grp >> 2) * 32 + (grp & 1) * 16 + ((grp >> 1) & 1) * 8;
        v_rows<FMT, D, 0>(s, [&](int run, u32x2 lo, u32x2 hi) {
          *reinterpret_cast<u32x2*>(dst + (32 * run) * S::VROW) = lo;
          *reinterpret_cast<u32x2*>(dst + (32 * run + 16) * S::VROW) = hi;
        });
      }
    } else {
#pragma unroll
      for (int n = 0; n < St::NK; ++n) {
        const int item = tid + n * TEAM, key = item / (D / 32), part = item % (D / 32);
        if (St::K_ITEMS % TEAM != 0 && item >= St::K_ITEMS) continue;
        uint8_t* dst = base + key * S::KROW + part * 64;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // NVFP4: two blocks in the run
          *reinterpret_cast<vec*>(dst + 16 * i) =
              decode8<FMT>(st.w[n * 5 + i], k_scale<FMT>(st.w[n * 5 + 4], i >> 1));
        }
      }
    }
  };
  auto bad_ids = [&]() {
    uint32_t bad = 0;
#pragma unroll
    for (int n = 0; n < St::NV; ++n) bad |= ((uint32_t)st.id[n] < n_pages ? 0u : 1u) << n;
    return bad;
  };

  // ---- the keys ---------------------------------------------------------------
  uint32_t bad = 0;  // V items of the staged step whose page is not in the cache
  int kt = k0, buf = 0;
  if (k0 < k1) {
    load_ids(kt);
    bad = bad_ids();
    load_bytes(kt);
    load_ids(kt + TILE_KEYS);
    decode(kt, 0, bad);
    bad = bad_ids();
    load_bytes(kt + TILE_KEYS);
    load_ids(kt + 2 * TILE_KEYS);
    __syncthreads();
  }
  for (; kt < k1; kt += TILE_KEYS, buf ^= 1) {
    const uint32_t ok = s_ok[(kt / TILE_KEYS) & 3];
    if (kt + TILE_KEYS < k1) {
      // the other buffer's step ended before the last barrier
      decode(kt + TILE_KEYS, buf ^ 1, bad);
      bad = bad_ids();
      load_bytes(kt + 2 * TILE_KEYS);  // (its flags: read two barriers from here, by then
      load_ids(kt + 3 * TILE_KEYS);    // those of two steps ago are done with)
    }
    const bool on = wave_on && kt <= pos_z && (p.window == 0 || kt + TILE_KEYS > pos_a - p.window + 1);
    if (on) {
      const uint8_t* kb = lds + buf * S::BYTES + col * S::KROW + half * 16;
      const uint8_t* vb = lds + buf * S::BYTES + S::V0 + col * S::VROW + half * 16;
      v16f x[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) x[u][r] = 0.0f;
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          x[u] = Wide<FMT>::mfma(*reinterpret_cast<const vec*>(kb + u * 32 * S::KROW + s * 32), qf[s], x[u]);
      const bool whole = __builtin_amdgcn_readfirstlane(ok) == 0x01010101u && kt + TILE_KEYS <= pos_a + 1 &&
                         kt + TILE_KEYS <= rg.hi && (p.window == 0 || kt > pos_z - p.window);
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int k = 32 * u + 8 * (r >> 2) + 4 * half + (r & 3), key = kt + k;
            if (!((ok >> (8 * (2 * u + (r >> 3)))) & 1) || key < see_lo || key >= see_hi)
              x[u][r] = -__builtin_inff();
          }
      }
      float t = x[0][0];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) t = fmaxf(t, x[u][r]);
      t = other_half_max(t);
      if (__any(t > lim)) {
        // (columns whose maximum stays keep it)
        const float mt = t > lim ? t : m;
        const float f = m > -__builtin_inff() ? __builtin_amdgcn_exp2f((m - mt) * cf) : 0.0f;
        m = mt;
        if (m > -__builtin_inff()) {
          lim = m + P_SLACK / cf;
          nb = P_BIAS - m * cf;
        }
        far = __any(fabsf(m * cf) > 0x1p20f && m > -__builtin_inff());
        z *= f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[i][r] *= f;
      }
      // 2^(x cf + nb): nb's rounding is a factor that all of a column's weights
      // share.  Where it could reach 1 the difference is taken first.
      float add = nb;
      if (far) {
        const float base = m > -__builtin_inff() ? m : 0.0f;
        add = P_BIAS;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r) x[u][r] -= base;
      }
      vec pb[4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
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
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          o[i] = Wide<FMT>::mfma(*reinterpret_cast<const vec*>(vb + i * 32 * S::VROW + e * 32), pb[e], o[i]);
    }
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
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const v4f t = {o[i][4 * r], o[i][4 * r + 1], o[i][4 * r + 2], o[i][4 * r + 3]};
        *reinterpret_cast<v4f*>(p.part_o + s * D + 32 * i + 8 * r + 4 * half) = t;
      }
    if (half == 0)
      p.part_ms[s] = make_float2(m * cf, z);
  }
}

template <int FMT, int D, int WAVES>
void launch(const AttnArgs& p, int tiles, int B, hipStream_t stream) {
  const dim3 grid((unsigned)(B * p.H), (unsigned)tiles, (unsigned)p.splits);
  hipLaunchKernelGGL((k_attn_tile<FMT, D, WAVES>), grid, dim3(64 * WAVES), 2 * TileLds<D>::BYTES,
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
