// Attention of the newest tokens of several sessions over one layer's block pool, for tiles of few rows.
//
//   o_t = sum_j softmax_j(scale q_t . k_j) v_j   over the keys j <= p_t, and j > p_t - window if there is one,
//
// the G query heads of a KV head and the tokens of a session packed into rows t G + g, NT * 8 rows to a tile. The
// sums run over the fp16 values that the pool reads back as (k_kvio.cu).
//
// What bounds it: every key and value is read once per tile, 4 d flops a row and key on data of d/2 .. 2 d bytes,
// so with up to 16 rows the pool's bytes from HBM. So nothing goes through shared memory: a warp takes whole
// 16-token pool blocks and loads them from global memory straight into the operands of m16n8k16 MMAs (the next
// block's keys once the scores are done, its values once the output is), and the rows are the 8 columns of the MMAs (S^T = K Q^T, O^T += V^T P^T), so
// that no MMA row is padding. That works without a transpose because the order of a contraction's index and of the output
// rows is free: lane (g, t) = (lane / 4, lane % 4) reads 16-byte runs of the key rows g and g + 8 at the
// dimensions that its quad's other lanes do not, and Q is loaded in the same order; of the value rows 2t, 2t+1,
// 2t+8, 2t+9 it reads the dimensions of column group g and pairs neighbouring rows with byte permutes.
//
// Softmax: base 2, the scores in fp32, a running maximum per row that is only raised when a score passes it by
// 2^8 or more (p in fp16 is scaled by 2^7, so it stays below 65504, and 2^-21 of the maximum is still a normal
// number); the sum adds the rounded p, so that the weights of the sum in fp32 are those of the products. One
// block per SM takes an equal share of all sessions' and heads' pool blocks, in order; a unit that is cut by the
// end of a share leaves (m, l, o) in a workspace, and the last of its blocks to arrive adds the parts in order,
// so the result does not depend on who was last.
#include <algorithm>

#include "kernels.h"

namespace mag {

namespace {

constexpr float kLazy = 8.0f;     // a score may pass the running maximum by 2^8
constexpr float kShift = 7.0f;    // p is scaled by 2^7

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// codes of bytes i, i + 1 (i = 0 or 2) of a word offset by 128 -> fp16 pair, exact
__device__ __forceinline__ __half2 s8_pair(uint32_t w, uint32_t sel) {
  return __hsub2(u32_as_h2(prmt(w, 0x64646464u, sel)), u32_as_h2(0x64806480u));
}
// One pool block (16 tokens of one head) as lane (g, t) holds it.
template <int D, int KV>
struct Raw {
  static constexpr int kRow = KV == 0 ? 2 * D : (KV == 1 ? D : D / 2);  // bytes of a vector
  static constexpr int KW = kRow / 4 / 4;   // words of a key row per lane (quad shares the row)
  static constexpr int VW = kRow / 8 / 4;   // words of a value row per lane (8 lanes share the row)
  uint32_t k[2][KW];   // key rows g, g + 8
  uint32_t v[4][VW];   // value rows 2t, 2t + 1, 2t + 8, 2t + 9
  uint32_t km[2];      // INT8: the row's scale (low half); INT4: (scale, min) of the lane's group
  uint32_t vm[KV == 2 ? 4 : 2];  // INT8: scales of rows (2t, 2t + 1), (2t + 8, 2t + 9); INT4: (scale, min) per row
};

template <int N>
__device__ __forceinline__ void ld_words(uint32_t (&w)[N], const uint8_t* p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = ldg_stream_u4(p + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = ldg_stream_u2(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = ldg_nc_u32(p);
  }
}

// kd: the block's K data of this head, km its scales.
template <int D, int KV>
__device__ __forceinline__ void load_k(Raw<D, KV>& r, const uint8_t* kd, const uint8_t* km, int g, int t) {
  using R = Raw<D, KV>;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* row = kd + (g + 8 * h) * R::kRow;
    if constexpr (KV == 0) {  // 16-byte runs, the quad's four side by side
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        uint32_t w[4];
        ld_words<4>(w, row + 64 * j + 16 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.k[h][4 * j + i] = w[i];
      }
    } else if constexpr (KV == 1) {
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        uint32_t w[4];
        ld_words<4>(w, row + 64 * j + 16 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.k[h][4 * j + i] = w[i];
      }
      r.km[h] = *reinterpret_cast<const uint16_t*>(km + 2 * (g + 8 * h));
    } else {
      ld_words<R::KW>(r.k[h], row + 4 * R::KW * t);
      r.km[h] = ldg_nc_u32(km + (g + 8 * h) * (D / 8) + 4 * (t * (D / 4) / 32));
    }
  }
}
// vd, vm: V data and scales. n_live: slots that hold tokens (value rows past them are taken as zero: a recycled
// block may hold anything there, and 0 times it must be 0).
template <int D, int KV>
__device__ __forceinline__ void load_v(Raw<D, KV>& r, const uint8_t* vd, const uint8_t* vm, int g, int t, int n_live) {
  using R = Raw<D, KV>;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int slot = 2 * t + (e & 1) + 8 * (e >> 1);
    const bool live = slot < n_live;
    const uint8_t* row = vd + slot * R::kRow;
    if constexpr (KV == 0) {  // 64 dimensions: 8 lanes' 16-byte runs side by side
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t w[4] = {0, 0, 0, 0};
        if (live) ld_words<4>(w, row + 128 * c + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.v[e][4 * c + i] = w[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < R::VW; ++i) r.v[e][i] = 0u;
      if (live) ld_words<R::VW>(r.v[e], row + 4 * R::VW * g);
      if constexpr (KV == 2) r.vm[e] = live ? ldg_nc_u32(vm + slot * (D / 8) + 4 * (g * (D / 8) / 32)) : 0u;
    }
  }
  if constexpr (KV == 1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t s = ldg_nc_u32(vm + 2 * (2 * t + 8 * h));
      if (2 * t + 8 * h >= n_live) s = 0;
      else if (2 * t + 8 * h + 1 >= n_live) s &= 0xFFFFu;
      r.vm[h] = s;
    }
  }
}

// Dimension of the first of the 8 consecutive values in chunk j of lane t's key-row share (and of Q's).
template <int D, int KV>
__device__ __forceinline__ constexpr int k_dim(int j, int t) {
  return KV == 0 ? 32 * j + 8 * t : (KV == 1 ? 64 * (j >> 1) + 16 * t + 8 * (j & 1) : (D / 4) * t + 8 * j);
}
// Dimension of output tile row g, m-tile i (16 dimensions: rows g and g + 8 of the MMA are its n = 2i, 2i + 1).
template <int D, int KV>
__device__ __forceinline__ constexpr int v_dim(int n, int g) {
  return KV == 0 ? 64 * (n >> 3) + 8 * g + (n & 7) : (D / 8) * g + n;
}

// The four 16-bit pairs of chunk j (8 consecutive dimensions) of a key row, in the MMA's order: FP16 and INT8
// pairs (0,1) (2,3) (4,5) (6,7), INT4 pairs (0,4) (1,5) (2,6) (3,7).
template <int D, int KV>
__device__ __forceinline__ void k_pairs(const uint32_t (&w)[Raw<D, KV>::KW], uint32_t km, int j, uint32_t (&o)[4]) {
  if constexpr (KV == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = w[4 * j + i];
  } else if constexpr (KV == 1) {
    const __half2 s = __low2half2(u32_as_h2(km));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = h2_as_u32(__hmul2(s8_pair(w[2 * j + (i >> 1)] ^ 0x80808080u, (i & 1) ? 0x4342 : 0x4140), s));
  } else {
    const __half2 s = __low2half2(u32_as_h2(km)), m = __high2half2(u32_as_h2(km));
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = h2_as_u32(__hfma2(u4_pair(w[j], i), s, m));
  }
}
// Value n (of D / 8) of the lane's column group for the row pair (a, b): fp16 (row a, row b).
template <int D, int KV>
__device__ __forceinline__ uint32_t v_pair(const uint32_t (&a)[Raw<D, KV>::VW], const uint32_t (&b)[Raw<D, KV>::VW],
                                           int n, __half2 s, __half2 m) {
  if constexpr (KV == 0) {
    return prmt(a[n >> 1], b[n >> 1], (n & 1) ? 0x7632 : 0x5410);
  } else if constexpr (KV == 1) {
    const uint32_t x = prmt(a[n >> 2] ^ 0x80808080u, b[n >> 2] ^ 0x80808080u, (n & 2) ? 0x7362 : 0x5140);
    return h2_as_u32(__hmul2(s8_pair(x, (n & 1) ? 0x4342 : 0x4140), s));
  } else {
    const uint32_t x = prmt(a[n >> 3], b[n >> 3], (n & 4) ? 0x7632 : 0x5410);
    return h2_as_u32(__hfma2(u4_pair(x, n & 3), s, m));
  }
}

// Warps of a block, one block per SM: as many as the registers of a warp's operands leave room for. FP16 holds 64
// registers of a pool block (in flight or in use), and 8 rows of o and Q another 48. INT8 and INT4 are bound by what these
// few warps hide: issue 48%, a quarter to a third of a warp's waits for loads, a quarter for fixed latencies.
template <int D, int KV, int NT>
constexpr int few_warps() {
  return D == 64 ? (KV == 0 && NT == 2 ? 12 : 16) : (KV == 0 ? (NT == 1 ? 12 : 8) : (NT == 1 ? 16 : 12));
}

template <int D, int NT, int W>
struct FewSmem {
  union {
    float o[W][NT * 8][D];
    float f[kAttendMaxShares][NT * 8];  // of a merge: the parts' factors
  };
  float ml[W][NT * 8][2];
  float inv[NT * 8];
  int last;
};

template <int D, int KV, int NT>
__global__ void __launch_bounds__(few_warps<D, KV, NT>() * 32, 1)
    attend_few_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ AttendShares sh) {
  constexpr int ROWS = NT * 8, NJ = D / 32, NM = D / 16, W = few_warps<D, KV, NT>(), T = W * 32;
  using R = Raw<D, KV>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  FewSmem<D, NT, W>& sm = *reinterpret_cast<FewSmem<D, NT, W>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const PoolGeom& P = a.pool;
  const int G = a.group;
  const int64_t data_part = (int64_t)P.n_kv_heads * 16 * R::kRow, meta_part = (int64_t)P.n_kv_heads * 16 * P.meta_bytes;
  const uint8_t* layer_base = P.base + (int64_t)a.layer * P.pool_blocks * P.block_bytes;

  // the block's share of all units' pool blocks, a piece of one unit at a time
  const int ue = sh.unit[blockIdx.x + 1], se = sh.step[blockIdx.x + 1];
  for (int u = sh.unit[blockIdx.x], s_first = sh.step[blockIdx.x]; u < ue || (u == ue && s_first < se);
       ++u, s_first = 0) {
    int si = 0;
    for (int i = 1; i < a.n_seg; ++i)
      if (u >= a.seg[i].unit0) si = i;
    const AttendSeg sg = a.seg[si];
    const int head = (u - sg.unit0) / sg.n_tiles, tile = u - sg.unit0 - head * sg.n_tiles;
    const int n_rows = sg.n_tok * G, r0 = tile * ROWS, live_rows = min(ROWS, n_rows - r0);
    int p_lo, p_hi, key0;
    const int n_steps = attend_unit_steps(sg.pos0, n_rows, G, a.window, r0, ROWS, 16, p_lo, p_hi, key0);
    const int s_end = u == ue ? se : n_steps;
    const int b0 = (key0 >> 4) + s_first, b1 = (key0 >> 4) + s_end;  // this piece's pool blocks
    const int len = sg.pos0 + sg.n_tok;                              // tokens in the cache
    const int32_t* table = P.tables + (int64_t)sg.sess * P.table_stride;

    // ids of the warp's blocks b0 + warp, + W, ..: 32 at a time
    int ids = 0, id_first = b0 + warp;
    auto fetch_ids = [&](int b) {
      const int bb = b + W * lane;
      ids = bb < b1 ? checked_block(table[bb], (int)P.pool_blocks, a.err) : 0;
      id_first = b;
    };
    R r;
    auto k_of = [&](int phys) { return layer_base + (int64_t)phys * P.block_bytes + (int64_t)head * 16 * R::kRow; };
    auto m_of = [&](int phys) {
      return layer_base + (int64_t)phys * P.block_bytes + 2 * data_part + (int64_t)head * 16 * P.meta_bytes;
    };
    int b = b0 + warp, phys = 0;
    if (b < b1) {
      fetch_ids(b);
      phys = __shfl_sync(0xffffffffu, ids, 0);
      load_k<D, KV>(r, k_of(phys), m_of(phys), g, t);
      load_v<D, KV>(r, k_of(phys) + data_part, m_of(phys) + meta_part, g, t, len - 16 * b);
    }

    // Q: row g of every 8-row column group, the dimensions in the key loads' order
    uint32_t qf[NT][NJ][4];
    int pos[NT][2];  // positions of this lane's score columns (rows 2t, 2t + 1)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int rr = r0 + 8 * n + g;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (rr < n_rows)
          w = ldg_stream_u4(a.q + (int64_t)(sg.row0 + rr / G) * a.ldq + (int64_t)(head * G + rr % G) * D +
                            k_dim<D, KV>(j, t));
        if constexpr (KV == 2) {
          qf[n][j][0] = prmt(w.x, w.z, 0x5410);
          qf[n][j][1] = prmt(w.x, w.z, 0x7632);
          qf[n][j][2] = prmt(w.y, w.w, 0x5410);
          qf[n][j][3] = prmt(w.y, w.w, 0x7632);
        } else {
          qf[n][j][0] = w.x, qf[n][j][1] = w.y, qf[n][j][2] = w.z, qf[n][j][3] = w.w;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) pos[n][c] = sg.pos0 + min(r0 + 8 * n + 2 * t + c, n_rows - 1) / G;
    }

    float o[NM][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) m[n][c] = -INFINITY, l[n][c] = 0.f;
    }

    for (; b < b1; b += W) {  // pool block b: keys 16 b .. 16 b + 15
      const int next = b + W;
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint32_t k0[4], k8[4];
        k_pairs<D, KV>(r.k[0], r.km[0], j, k0);
        k_pairs<D, KV>(r.k[1], r.km[1], j, k8);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_16816(s[n], k0[0], k8[0], k0[1], k8[1], qf[n][j][0], qf[n][j][1]);
          mma_16816(s[n], k0[2], k8[2], k0[3], k8[3], qf[n][j][2], qf[n][j][3]);
        }
      }
      // the keys' registers are free: the next block's
      if (next < b1) {
        if (next - id_first >= W * 32) fetch_ids(next);
        phys = __shfl_sync(0xffffffffu, ids, (next - id_first) / W);
        load_k<D, KV>(r, k_of(phys), m_of(phys), g, t);
      }
      // scale (base 2), mask; element (c, h) of column group n: key 16 b + g + 8 h, row 8 n + 2 t + c
      const bool inside = 16 * b + 15 <= p_lo && (!a.window || 16 * b > p_hi - a.window);
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[n][e] * a.scale_log2;
          if (!inside) {
            const int back = pos[n][e & 1] - (16 * b + g + 8 * (e >> 1));
            if (back < 0 || (a.window && back >= a.window)) x = -INFINITY;
          }
          s[n][e] = x;
          raise |= x >= m[n][e & 1] + kLazy;  // 2^26 and more from zero one step of fp32 is 8 or more
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaxf(s[n][c], s[n][c + 2]);
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
            const float mn = fmaxf(m[n][c], x);
            const float f = m[n][c] == -INFINITY ? 0.f : ex2(m[n][c] - mn);
            l[n][c] *= f;
            m[n][c] = mn;
#pragma unroll
            for (int i = 0; i < NM; ++i) {
              o[i][n][c] *= f;
              o[i][n][c + 2] *= f;
            }
          }
      }
      uint32_t p0[NT], p1[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = ex2(s[n][e] - (m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1] - kShift));
        const __half2 h0 = __floats2half2_rn(p[0], p[1]), h1 = __floats2half2_rn(p[2], p[3]);
        const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
        l[n][0] += f0.x + f1.x;
        l[n][1] += f0.y + f1.y;
        p0[n] = movmatrix_t(h2_as_u32(h0));  // keys 2t, 2t + 1 of row g
        p1[n] = movmatrix_t(h2_as_u32(h1));  // keys 2t + 8, 2t + 9
      }
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        __half2 sa = {}, ma = {}, sb = {}, mb = {};
        if constexpr (KV == 1) {
          sa = u32_as_h2(r.vm[0]);
          sb = u32_as_h2(r.vm[1]);
        } else if constexpr (KV == 2) {
          sa = u32_as_h2(prmt(r.vm[0], r.vm[1], 0x5410)), ma = u32_as_h2(prmt(r.vm[0], r.vm[1], 0x7632));
          sb = u32_as_h2(prmt(r.vm[2], r.vm[3], 0x5410)), mb = u32_as_h2(prmt(r.vm[2], r.vm[3], 0x7632));
        }
        const uint32_t a0 = v_pair<D, KV>(r.v[0], r.v[1], 2 * i, sa, ma), a1 = v_pair<D, KV>(r.v[0], r.v[1], 2 * i + 1, sa, ma);
        const uint32_t a2 = v_pair<D, KV>(r.v[2], r.v[3], 2 * i, sb, mb), a3 = v_pair<D, KV>(r.v[2], r.v[3], 2 * i + 1, sb, mb);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_16816(o[i][n], a0, a1, a2, a3, p0[n], p1[n]);
      }
      if (next < b1) load_v<D, KV>(r, k_of(phys) + data_part, m_of(phys) + meta_part, g, t, len - 16 * next);
    }

    // ---- the warps' results
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], k);
        const int row = 8 * n + 2 * t + c;
        if (g == 0) sm.ml[warp][row][0] = m[n][c], sm.ml[warp][row][1] = l[n][c];
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          sm.o[warp][row][v_dim<D, KV>(2 * i, g)] = o[i][n][c];
          sm.o[warp][row][v_dim<D, KV>(2 * i + 1, g)] = o[i][n][c + 2];
        }
      }
    }
    __syncthreads();
    auto out_at = [&](int row) {
      const int rr = r0 + row;
      return a.o + (int64_t)(sg.row0 + rr / G) * a.ldo + (int64_t)(head * G + rr % G) * D;
    };
    // every warp with work left its (m, l, o); warps without have m = -inf, l = 0, o = 0
    const bool whole = s_first == 0 && s_end == n_steps;
    const int mine = 2 * (int)blockIdx.x + (u == sh.unit[blockIdx.x] ? 0 : 1);
    for (int e = threadIdx.x; e < live_rows * (D / 4); e += T) {
      const int row = e / (D / 4), c4 = e % (D / 4);
      float mx = sm.ml[0][row][0];
#pragma unroll
      for (int w = 1; w < W; ++w) mx = fmaxf(mx, sm.ml[w][row][0]);
      float ls = 0.f;
      float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = sm.ml[w][row][0] == -INFINITY ? 0.f : ex2(sm.ml[w][row][0] - mx);
        const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][row][4 * c4]);
        ls = fmaf(f, sm.ml[w][row][1], ls);
        os.x = fmaf(f, x.x, os.x), os.y = fmaf(f, x.y, os.y), os.z = fmaf(f, x.z, os.z), os.w = fmaf(f, x.w, os.w);
      }
      if (whole) {
        const float inv = 1.0f / ls;
        uint2 h;
        h.x = h2_as_u32(__floats2half2_rn(os.x * inv, os.y * inv));
        h.y = h2_as_u32(__floats2half2_rn(os.z * inv, os.w * inv));
        *reinterpret_cast<uint2*>(out_at(row) + 4 * c4) = h;
      } else {
        __stcg(reinterpret_cast<float4*>(a.part + ((int64_t)mine * ROWS + row) * D) + c4, os);
        if (c4 == 0) __stcg(reinterpret_cast<float2*>(a.part_ml) + (int64_t)mine * ROWS + row, make_float2(mx, ls));
      }
    }
    if (whole) {
      __syncthreads();  // the shared results are read before the next piece's
      continue;
    }
    // ---- a cut unit: the last of its blocks to arrive adds the parts in order
    __threadfence();
    int c0 = blockIdx.x, c1 = blockIdx.x;  // the blocks that share it
    while (sh.unit[c0] == u && sh.step[c0] > 0) --c0;
    while (sh.unit[c1 + 1] == u && sh.step[c1 + 1] < n_steps) ++c1;
    __syncthreads();
    if (threadIdx.x == 0) {
      const uint32_t prev = atomicAdd(a.arrivals + c0, 1u);
      sm.last = (int)prev == c1 - c0;
      if (sm.last) a.arrivals[c0] = 0;  // for the next launch
    }
    __syncthreads();
    if (!sm.last) continue;
    __threadfence();
    const int n_parts = c1 - c0 + 1;
    auto slot_of = [&](int c) { return 2 * c + (u == sh.unit[c] ? 0 : 1); };
    // a warp per row: the parts' factors over the row's sum
    for (int row = warp; row < live_rows; row += W) {
      const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
      float mt = -INFINITY;
      for (int k = lane; k < n_parts; k += 32) mt = fmaxf(mt, __ldcg(ml + (int64_t)slot_of(c0 + k) * ROWS + row).x);
      mt = warp_max(mt);
      float lt = 0.f;
      for (int k = lane; k < n_parts; k += 32) {
        const float2 x = __ldcg(ml + (int64_t)slot_of(c0 + k) * ROWS + row);
        const float f = x.x == -INFINITY ? 0.f : ex2(x.x - mt);
        sm.f[k][row] = f;
        lt = fmaf(f, x.y, lt);
      }
      lt = warp_sum(lt);
      if (lane == 0) sm.inv[row] = 1.0f / lt;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < live_rows * (D / 4); e += T) {
      const int row = e / (D / 4), c4 = e % (D / 4);
      float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int k = 0; k < n_parts; ++k) {
        const float f = sm.f[k][row];
        const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part + ((int64_t)slot_of(c0 + k) * ROWS + row) * D) + c4);
        os.x = fmaf(f, x.x, os.x), os.y = fmaf(f, x.y, os.y), os.z = fmaf(f, x.z, os.z), os.w = fmaf(f, x.w, os.w);
      }
      const float inv = sm.inv[row];
      uint2 h;
      h.x = h2_as_u32(__floats2half2_rn(os.x * inv, os.y * inv));
      h.y = h2_as_u32(__floats2half2_rn(os.z * inv, os.w * inv));
      *reinterpret_cast<uint2*>(out_at(row) + 4 * c4) = h;
    }
    __syncthreads();
  }
}

template <int D, int KV, int NT>
cudaError_t launch_few_t(const Launch& L, const AttendArgs& a, const AttendShares& sh) {
  constexpr int W = few_warps<D, KV, NT>(), smem = sizeof(FewSmem<D, NT, W>);
  cudaError_t e = cudaFuncSetAttribute(attend_few_kernel<D, KV, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(L, attend_few_kernel<D, KV, NT>, dim3(sh.n), dim3(W * 32), smem, a, sh);
}
template <int D, int KV>
cudaError_t launch_few_nt(const Launch& L, const AttendArgs& a, const AttendShares& sh, int tile_rows) {
  return tile_rows == 8 ? launch_few_t<D, KV, 1>(L, a, sh) : launch_few_t<D, KV, 2>(L, a, sh);
}
template <int D>
cudaError_t launch_few_kv(const Launch& L, const AttendArgs& a, const AttendShares& sh, int tile_rows) {
  switch (a.pool.kv_dtype) {
    case 0: return launch_few_nt<D, 0>(L, a, sh, tile_rows);
    case 1: return launch_few_nt<D, 1>(L, a, sh, tile_rows);
    default: return launch_few_nt<D, 2>(L, a, sh, tile_rows);
  }
}

}  // namespace

// The sessions' units, and every block's share of their steps, in order. Equal shares, block b beginning at step
// total b / n, keep every SM busy to the end, but most blocks then work on two units or more; where there are no more
// units than blocks and whole parts of units take a block at most `piece` steps longer, it gets one part of one unit.
void attend_shares(AttendArgs& a, int tile_rows, int step_keys, int max_blocks, int min_steps, int piece,
                   AttendShares& sh) {
  int64_t total = 0, units = 0;
  int p_lo, p_hi, key0;
  auto steps = [&](const AttendSeg& s, int tile) {
    return attend_unit_steps(s.pos0, s.n_tok * a.group, a.group, a.window, tile * tile_rows, tile_rows, step_keys, p_lo,
                             p_hi, key0);
  };
  max_blocks = std::min(max_blocks, kAttendMaxShares);
  int64_t per_head[MAG_MAX_BATCH];
  int most = 1;
  for (int i = 0; i < a.n_seg; ++i) {
    AttendSeg& s = a.seg[i];
    s.n_tiles = (int)(((int64_t)s.n_tok * a.group + tile_rows - 1) / tile_rows);
    s.unit0 = (int32_t)units;
    units += (int64_t)s.n_tiles * a.n_kv_heads;
    per_head[i] = 0;
    for (int j = 0; j < s.n_tiles; ++j) {
      const int n = steps(s, j);
      per_head[i] += n;
      most = std::max(most, n);
    }
    total += per_head[i] * a.n_kv_heads;
  }
  a.n_units = (int32_t)units;
  const int64_t equal = std::max<int64_t>(min_steps, (total + max_blocks - 1) / max_blocks);
  if (units <= max_blocks) {
    // the shortest parts, all of a unit alike, that make no more blocks than there may be
    auto blocks = [&](int64_t len) {
      int64_t n = 0;
      for (int i = 0; i < a.n_seg; ++i)
        for (int j = 0; j < a.seg[i].n_tiles; ++j) n += (steps(a.seg[i], j) + len - 1) / len * a.n_kv_heads;
      return n;
    };
    int64_t lo = std::min<int64_t>(min_steps, most), hi = most;  // hi: one part a unit
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (blocks(mid) <= max_blocks) hi = mid;
      else lo = mid + 1;
    }
    if (lo <= equal + piece) {
      int b = 0;
      for (int i = 0; i < a.n_seg; ++i)
        for (int h = 0; h < a.n_kv_heads; ++h)
          for (int j = 0; j < a.seg[i].n_tiles; ++j) {
            const int64_t n = steps(a.seg[i], j), parts = (n + lo - 1) / lo;
            for (int64_t k = 0; k < parts; ++k, ++b) {
              sh.unit[b] = a.seg[i].unit0 + h * a.seg[i].n_tiles + j;
              sh.step[b] = (int32_t)(n * k / parts);
            }
          }
      sh.n = b;
      sh.unit[b] = a.n_units;
      sh.step[b] = 0;
      return;
    }
  }
  sh.n = (int32_t)std::max<int64_t>(1, std::min<int64_t>(max_blocks, (total + min_steps - 1) / min_steps));
  int si = 0, head = 0, tile = 0;
  int64_t at = 0;
  for (int b = 0; b < sh.n; ++b) {
    const int64_t want = total * b / sh.n;
    while (true) {
      const AttendSeg& s = a.seg[si];
      if (tile == 0 && at + per_head[si] <= want) {  // a whole head further
        at += per_head[si];
        if (++head == a.n_kv_heads) head = 0, ++si;
        continue;
      }
      const int n = steps(s, tile);
      if (at + n > want) break;
      at += n;
      if (++tile == s.n_tiles) {
        tile = 0;
        if (++head == a.n_kv_heads) head = 0, ++si;
      }
    }
    sh.unit[b] = a.seg[si].unit0 + head * a.seg[si].n_tiles + tile;
    sh.step[b] = (int32_t)(want - at);
  }
  sh.unit[sh.n] = a.n_units;
  sh.step[sh.n] = 0;
}

cudaError_t launch_attend_few(const Launch& L, AttendArgs& a, int n_sm, int tile_rows) {
  if (a.n_seg < 1 || a.n_seg > MAG_MAX_BATCH || (tile_rows != 8 && tile_rows != 16)) return cudaErrorInvalidValue;
  // a block's share is at least a pool block for each of (about) its warps
  AttendShares sh;
  attend_shares(a, tile_rows, 16, n_sm, 12, 24, sh);
  return a.pool.head_dim == 64 ? launch_few_kv<64>(L, a, sh, tile_rows) : launch_few_kv<128>(L, a, sh, tile_rows);
}

}  // namespace mag
