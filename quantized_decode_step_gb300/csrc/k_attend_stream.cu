// Attention of the newest tokens of several sessions over one layer's block pool, for 17 to 128 packed rows: tcgen05, one
// tile of rows, the keys in two streams.
//
//   o_t = sum_j softmax_j(scale q_t . k_j) v_j   over the keys j <= p_t, and j > p_t - window if there is one.
//
// What bounds it: K and V are read once for all rows, so the loads, and the chain from a step's scores to its products. A
// block takes a step of 128 keys (of either stream) in 1.8 us of FP16, 0.8 of the copy rate over 152 blocks, and in 2.25
// of INT8 and 1.75 of INT4, where it is the chain: issue 36%, the warps' waits mostly loads (28%) and instruction
// fetch (18%). A call takes about 12 us besides, for its start and the merge. A 128-row MMA tile is mostly padding with few
// rows, but the tensor core has the time, and everything that costs instructions is done once: the expansion of INT8 and
// INT4 by eight warps of their own, the softmax by the one warp per stream and 32 rows that has any. Up to 16 rows the
// register kernel reads the keys once as well and is faster; beyond, and from where on the two-tile kernel is: ops.cu.
//
// Even and odd steps of 128 keys are two streams with a maximum, a sum and an o each, so that one's softmax runs while
// the tensor core has the other's products; they are joined at the end, in tensor memory. Roles, the softmax's base and
// lazy maximum and the shares of the units' steps are those of k_attend_tc.cu; the sum adds the rounded p, as the register
// kernel does. INT4 values are left in the order that their expansion makes them in (0, 4, 1, 5, 2, 6, 3, 7 of every
// eight): of K it only has to be Q's, of V it is undone as o is stored.
#include <algorithm>

#include "attend_tc.cuh"

namespace mag {

namespace {

using namespace tc;

// The ring of K and V tiles (fp16, 128 keys, 128-byte swizzled halves of 64 dimensions) in shared memory.
// FP16: a loader warp fills it by TMA. INT8, INT4: kExpand warps copy the stored bytes into slots of their own, kRaw
// tiles ahead, each thread the 16-byte runs that it expands later, so that no thread waits for another's copies
// (128 rows over 20,000 INT4 keys: 33.6 us; 37.5 with a loader warp that issues a bulk copy per pool block). Tiles come and
// go in the order of in_order().
template <int D, int KV>
struct RingShape {
  static constexpr int kTile = kKeys * D * 2, kHalf = kKeys * 128;
  static constexpr int kStages = D == 128 ? (KV == 0 ? 6 : 4) : 8;
  static constexpr int kRowB = KV == 0 ? 2 * D : (KV == 1 ? D : D / 2), kMetaB = KV == 0 ? 0 : (KV == 1 ? 2 : D / 8);
  static constexpr int kExpand = KV == 0 ? 0 : 8;  // expanding warps
  static constexpr int kRuns = kRowB / 16;         // 16-byte runs of a stored row
  static constexpr int kItems = KV == 0 ? 1 : kKeys * kRuns / (32 * 8);  // runs of a thread and tile
  static constexpr int kRawBytes = KV == 0 ? 0 : kItems * 256 * 20;      // of a tile: a run and 4 bytes of its metadata each
  static constexpr int kRaw = KV == 0 ? 0 : (kItems == 4 ? 3 : 6);
  static constexpr int kThreads = (12 + kExpand) * 32;
  static constexpr int kBytes = kStages * kTile + kRaw * kRawBytes, kBars = 2 * kStages;
};
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {  // zeros where it is not
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}

// The order in which a piece's tiles are loaded, expanded and used: K 0, K 1, then V j, K j + 2 for every step j.
// f(step, part) with part 0 for K.
template <typename F>
__device__ __forceinline__ bool in_order(int s0, int s1, F f) {
  if (!f(s0, 0)) return false;
  if (s0 + 1 < s1 && !f(s0 + 1, 0)) return false;
  for (int s = s0; s < s1; ++s) {
    if (!f(s, 1)) return false;
    if (s + 2 < s1 && !f(s + 2, 0)) return false;
  }
  return true;
}

template <int D, int KV>
struct Ring : RingShape<D, KV> {
  using S = RingShape<D, KV>;
  uint8_t *tiles, *raw;
  uint64_t *full, *empty;
  __device__ Ring(uint8_t* mem, uint64_t* bars)
      : tiles(mem), raw(mem + S::kStages * S::kTile), full(bars), empty(full + S::kStages) {}
  __device__ void init() const {
    for (int i = 0; i < S::kStages; ++i) {
      mb_init(full + i, KV == 0 ? 1 : S::kExpand);
      mb_init(empty + i, 1);
    }
  }

  // FP16's loader warp: share(f) calls f(session, head, first key, first step, end step) for every piece.
  template <typename Share>
  __device__ void load(const CUtensorMap& map, const AttendArgs& a, Share share) const {
    const int lane = threadIdx.x & 31;
    const PoolGeom& P = a.pool;
    const uint8_t* layer_base = P.base + (int64_t)a.layer * P.pool_blocks * P.block_bytes;
    const int64_t data_part = (int64_t)P.n_kv_heads * 16 * S::kRowB;
    int g = 0;
    share([&](const AttendSeg& sg, int head, int key0, int s0, int s1) {
      const int32_t* table = P.tables + (int64_t)sg.sess * P.table_stride;
      const int len = sg.pos0 + sg.n_tok, n_blk = (len + 15) >> 4;
      // block ids, one a lane: of four steps from `at` on; V comes two steps after K, so two such windows
      int ids[2] = {0, 0}, at[2] = {-4, -4};
      return in_order(s0, s1, [&](int s, int part) {
        const int key = key0 + s * kKeys, b0 = key >> 4;
        if (s >= at[part] + 4 || at[part] < s0) {
          const int b = b0 + lane;
          ids[part] = b < n_blk ? checked_block(table[b], (int)P.pool_blocks, a.err) : 0;
          at[part] = s;
        }
        const int nb = min(8, n_blk - b0);        // pool blocks of this step
        const int nv = min(8, (len - key) >> 4);  // of them, whole ones
        const int id_w = ids[part], id_at = (s - at[part]) * 8;
        const int my = __shfl_sync(0xffffffffu, id_w, id_at + (lane & 7));
        const int st = g % S::kStages;
        if (g >= S::kStages && !mb_wait_warp(empty + st, ((g / S::kStages) - 1) & 1, a.wait_limit)) {
          if (lane == 0) atomicOr(a.err, kErrAttend);
          return false;
        }
        uint8_t* tile = tiles + st * S::kTile;
        int n_tma = nb;
        if (part == 1 && nv < 8) {
          // the step that holds the session's end: value rows past it are zeros (a slot there may hold anything, and 0
          // times it must be 0), the block it lies in is copied row by row
          n_tma = nv;
          const int y0 = nv * 16;
          for (int i = lane; i < (kKeys - y0) * (D / 8); i += 32) {  // a multiple of 32
            const int row = y0 + i / (D / 8), c = i % (D / 8);
            uint4 w = make_uint4(0, 0, 0, 0);
            const int b = __shfl_sync(0xffffffffu, id_w, id_at + (row >> 4));
            if (key + row < len)
              w = *reinterpret_cast<const uint4*>(layer_base + (int64_t)b * P.block_bytes + data_part +
                                                  ((int64_t)head * 16 + (row & 15)) * S::kRowB + 16 * c);
            *reinterpret_cast<uint4*>(tile + (c >> 3) * S::kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = w;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        if (lane == 0) mb_expect(full + st, (uint32_t)n_tma * 16 * D * 2);
        __syncwarp();
        const int blk = lane & 7, half = lane >> 3;
        if (blk < n_tma && half < D / 64)
          tma_3d(su32(tile) + half * S::kHalf + blk * 2048, &map, half * 64, (part * P.n_kv_heads + head) * 16, my, full + st);
        ++g;
        return true;
      });
    });
    // leave no copy in flight, also when a consumer gave up and will not wait for it
    for (int f = max(0, g - S::kStages); f < g; ++f) mb_wait(full + f % S::kStages, (f / S::kStages) & 1);
  }

  // Expanding warp w of kExpand: copies tile g, then expands the one kRaw - 1 before it.
  template <typename Share>
  __device__ void expand(int w, const AttendArgs& a, Share share) const {
    const int lane = threadIdx.x & 31, thread = w * 32 + lane;
    const PoolGeom& P = a.pool;
    const int64_t data_part = (int64_t)P.n_kv_heads * 16 * S::kRowB, meta_part = (int64_t)P.n_kv_heads * 16 * S::kMetaB;
    // A warp's 32 runs are whole stored rows. Of 8 lanes side by side each writes another 16 bytes of the 128-byte
    // swizzled rows: with two (INT8) or four (INT4) fp16 runs a lane that takes two rows, or four.
    constexpr int kRq = KV == 1 ? 2 : 4, kRunQ = 8 / kRq, kQr = S::kRuns / kRunQ, kRowsW = 32 / S::kRuns;
    const int run = (lane / kRq) % kRunQ + kRunQ * ((lane >> 3) % kQr);
    const int row_w = (lane & (kRq - 1)) + kRq * ((lane >> 3) / kQr) + w * kRowsW;  // of item 0; 8 kRowsW further an item
    const uint8_t* src0 = P.base + (int64_t)a.layer * P.pool_blocks * P.block_bytes;
    const uint8_t* data0 = src0 + (row_w & 15) * S::kRowB + 16 * run;
    const uint8_t* meta0 = src0 + 2 * data_part + (KV == 1 ? (row_w & 14) * 2 : (row_w & 15) * S::kMetaB + 4 * run);
    const uint32_t raw16 = su32(raw) + thread * 16, raw4 = su32(raw) + S::kItems * 256 * 16 + thread * 4;
    int g = 0;   // tiles copied
    int ge = 0;  // and expanded
    auto expand_next = [&] {
      const int st = ge % S::kStages, r = ge % S::kRaw;
      if (ge >= S::kStages && !mb_wait_warp(empty + st, ((ge / S::kStages) - 1) & 1, a.wait_limit)) {
        if (lane == 0) atomicOr(a.err, kErrAttend);
        return false;
      }
      const uint8_t* src = raw + r * S::kRawBytes;
#pragma unroll
      for (int i = 0; i < S::kItems; ++i) {
        const int row = row_w + i * 8 * kRowsW;
        const uint4 c = *reinterpret_cast<const uint4*>(src + (i * 256 + thread) * 16);
        uint32_t meta = *reinterpret_cast<const uint32_t*>(src + S::kItems * 256 * 16 + (i * 256 + thread) * 4);
        if (KV == 1 && (row & 1)) meta >>= 16;
        const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
        const __half2 sc = __low2half2(u32_as_h2(meta)), mn = __high2half2(u32_as_h2(meta));
        uint8_t* row_p = tiles + st * S::kTile + row * 128;
        if constexpr (KV == 1) {  // 16 values: two runs of 8
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t h = __byte_perm(cw[2 * e + (k >> 1)] ^ 0x80808080u, 0x64646464u, (k & 1) ? 0x4342 : 0x4140);
              v[k] = h2_as_u32(__hmul2(__hsub2(u32_as_h2(h), u32_as_h2(0x64806480u)), sc));
            }
            const int cc = 2 * run + e;
            *reinterpret_cast<uint4*>(row_p + (cc >> 3) * S::kHalf + (((cc & 7) ^ (row & 7)) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
        } else {  // 32 values: four runs of 8, pairs (i, i + 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] = h2_as_u32(__hfma2(u4_pair(cw[e], k), sc, mn));
            const int cc = 4 * run + e;
            *reinterpret_cast<uint4*>(row_p + (cc >> 3) * S::kHalf + (((cc & 7) ^ (row & 7)) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mb_arrive(full + st);
      ++ge;
      return true;
    };
    bool ok = true;
    share([&](const AttendSeg& sg, int head, int key0, int s0, int s1) {
      const int32_t* table = P.tables + (int64_t)sg.sess * P.table_stride;
      const int len = sg.pos0 + sg.n_tok, n_blk = (len + 15) >> 4;
      // block ids, one a lane: of four steps from `at` on, and of the next four; V comes two steps after K
      auto ids_at = [&](int s) {
        const int b = ((key0 + s * kKeys) >> 4) + lane;
        return b < n_blk ? table[b] : 0;
      };
      int ids[2], next[2], at[2] = {s0, s0};
      ids[0] = ids[1] = checked_block(ids_at(s0), (int)P.pool_blocks, a.err);
      next[0] = next[1] = ids_at(s0 + 4);
      const uint8_t* data_h = data0 + (int64_t)head * 16 * S::kRowB;
      const uint8_t* meta_h = meta0 + (int64_t)head * 16 * S::kMetaB;
      ok = in_order(s0, s1, [&](int s, int part) {
        if (s >= at[part] + 4) {
          ids[part] = checked_block(next[part], (int)P.pool_blocks, a.err);
          next[part] = ids_at(s + 4);
          at[part] = s;
        }
        const int live = len - (key0 + s * kKeys);  // rows that hold tokens; the others become zeros
        const uint32_t slot = (uint32_t)(g % S::kRaw) * S::kRawBytes;
        const int my_ids = ids[part], id_at = (s - at[part]) * 8;
#pragma unroll
        for (int i = 0; i < S::kItems; ++i) {
          const int row = row_w + i * 8 * kRowsW;
          const int64_t blk = (int64_t)__shfl_sync(0xffffffffu, my_ids, id_at + (row >> 4)) * P.block_bytes;
          copy16(raw16 + slot + i * 256 * 16, data_h + blk + part * data_part, row < live);
          copy4(raw4 + slot + i * 256 * 4, meta_h + blk + part * meta_part, row < live);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++g < S::kRaw) return true;
        asm volatile("cp.async.wait_group %0;" ::"n"(S::kRaw - 1) : "memory");
        return expand_next();
      });
      return ok;
    });
    asm volatile("cp.async.wait_all;" ::: "memory");
    while (ok && ge < g) ok = expand_next();
  }
};

// Dimension of column c (of o, of a value row): INT4 leaves every eight in its expansion's order.
template <int KV>
__device__ __forceinline__ constexpr int dim_of(int c) {
  return KV == 2 ? (c & ~7) | ((c & 1) * 4 + ((c & 7) >> 1)) : c;
}
// 8 fp16 values in that order.
template <int KV>
__device__ __forceinline__ uint4 in_expansion_order(const uint4& w) {
  return KV == 2 ? make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632), __byte_perm(w.y, w.w, 0x5410),
                              __byte_perm(w.y, w.w, 0x7632))
                 : w;
}

// One tile of up to 128 packed rows of a session and KV head over its keys.
struct Unit {
  AttendSeg sg;
  int head, r0, n_rows, live;  // first packed row, rows of the session, rows of the tile
  int p_lo, p_hi, key0, n_steps;
};
__device__ __forceinline__ Unit unit_of(const AttendArgs& a, int u) {
  Unit x;
  int si = 0;
  for (int i = 1; i < a.n_seg; ++i)
    if (u >= a.seg[i].unit0) si = i;
  x.sg = a.seg[si];
  const int v = u - x.sg.unit0;
  x.head = v / x.sg.n_tiles;
  x.r0 = (v - x.head * x.sg.n_tiles) * kRows;
  x.n_rows = x.sg.n_tok * a.group;
  x.live = min(kRows, x.n_rows - x.r0);
  x.n_steps = attend_unit_steps(x.sg.pos0, x.n_rows, a.group, a.window, x.r0, kRows, kKeys, x.p_lo, x.p_hi, x.key0);
  return x;
}
// f(unit, index, first step, end step) for every piece of this block's share.
template <typename F>
__device__ __forceinline__ void for_share(const AttendArgs& a, const AttendShares& sh, F f) {
  int u = sh.unit[blockIdx.x], s = sh.step[blockIdx.x];
  const int ue = sh.unit[blockIdx.x + 1], se = sh.step[blockIdx.x + 1];
  while (u < ue || (u == ue && s < se)) {
    const Unit x = unit_of(a, u);
    if (!f(x, u, s, u == ue ? se : x.n_steps)) return;
    ++u;
    s = 0;
  }
}


template <int D, int KV>
struct Cfg : RingShape<D, KV> {
  using R = RingShape<D, KV>;
  static constexpr int kBars = R::kBars + 9;
  static constexpr int kSmem = R::kTile + R::kBytes + kRows * 8 + kBars * 8 + 64 + 1024;
};

// 8 columns as fp16 in the order of their dimensions.
template <int KV>
__device__ __forceinline__ uint4 pack8(const float (&o)[8]) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[dim_of<KV>(i)] = o[i];
  return make_uint4(h2_as_u32(__floats2half2_rn(x[0], x[1])), h2_as_u32(__floats2half2_rn(x[2], x[3])),
                    h2_as_u32(__floats2half2_rn(x[4], x[5])), h2_as_u32(__floats2half2_rn(x[6], x[7])));
}

template <int D, int KV>
__global__ void __launch_bounds__(Cfg<D, KV>::kThreads, 1)
    attend_stream_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ AttendArgs a,
                         const __grid_constant__ AttendShares sh) {
  using C = Cfg<D, KV>;
  constexpr uint32_t kIdescQK = (1u << 4) | ((uint32_t)(kKeys >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
  constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;
  float2* ml_b = reinterpret_cast<float2*>(smem + C::kTile + C::kBytes);  // the second stream's (m, l)
  uint64_t* bars = reinterpret_cast<uint64_t*>(ml_b + kRows);
  const Ring<D, KV> ring(smem + C::kTile, bars);
  uint64_t* q_full = bars + C::R::kBars;
  uint64_t* s_full = q_full + 1;   // [2]: S of the stream is in tensor memory (and o holds its earlier steps)
  uint64_t* p_full = s_full + 2;   // [2]: P is
  uint64_t* o_full = p_full + 2;   // [2]: o is final
  uint64_t* joined = o_full + 2;   // the eight softmax warps
  uint64_t* mma_done = joined + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ring.init();
    mb_init(q_full, 8);
    for (int i = 0; i < 2; ++i) {
      mb_init(s_full + i, 1);
      mb_init(p_full + i, 4);
      mb_init(o_full + i, 1);
    }
    mb_init(joined, 8);
    mb_init(mma_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tm_s = tmem, tm_o = tmem + 2 * kKeys;  // S (and P) of stream t at + 128 t, o of stream t at + 128 t

  pdl_trigger();  // the merge kernel may be put in place; it waits for this grid's end
  if (warp == 0) {
    if constexpr (KV == 0) ring.load(map, a, [&](auto f) {
      for_share(a, sh, [&](const Unit& x, int, int s0, int s1) { return f(x.sg, x.head, x.key0, s0, s1); });
    });
  } else if (warp == 1) {
    if (lane == 0) {
      // ---- MMA issuer
      int g = 0, piece = 0, cnt[2] = {0, 0};
      const uint32_t q_a = su32(q_s), ring_a = su32(ring.tiles);
      for_share(a, sh, [&](const Unit&, int, int s0, int s1) {
        bool ok = mb_wait(q_full, piece & 1, a.wait_limit);
        ++piece;
        ok = ok && in_order(s0, s1, [&](int s, int part) {
          const int t = (s - s0) & 1, st = g % C::kStages;
          if (!mb_wait(ring.full + st, (g / C::kStages) & 1, a.wait_limit)) return false;
          if (part == 0) {
            tc_after();
            const uint64_t qd = smem_desc(q_a, 16), kd = smem_desc(ring_a + st * C::kTile, 16);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint64_t off = (uint64_t)((k >> 2) * C::kHalf + (k & 3) * 32) >> 4;
              mma_ss(tm_s + t * kKeys, qd + off, kd + off, kIdescQK, k != 0);
            }
            mma_commit(s_full + t);
          } else {
            if (!mb_wait(p_full + t, cnt[t] & 1, a.wait_limit)) return false;
            ++cnt[t];
            tc_after();
            const uint64_t vd = smem_desc(ring_a + st * C::kTile, C::kHalf);
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_ts(tm_o + t * 128, tm_s + t * kKeys + k * 8, vd + ((uint64_t)(k * 2048) >> 4), kIdescPV,
                     (s - s0 > 1) || k != 0);
            if (s + 2 >= s1) mma_commit(o_full + t);
          }
          mma_commit(ring.empty + st);
          ++g;
          return true;
        });
        if (!ok) atomicOr(a.err, kErrAttend);
        return ok;
      });
      // every MMA has completed before the block frees its tensor memory
      mma_commit(mma_done);
      mb_wait(mma_done, 0);
    }
  } else if (warp >= 12) {
    if constexpr (KV != 0)
      ring.expand(warp - 12, a, [&](auto f) {
        for_share(a, sh, [&](const Unit& x, int, int s0, int s1) { return f(x.sg, x.head, x.key0, s0, s1); });
      });
  } else if (warp >= 4) {
    // ---- softmax of stream t, one row a thread
    const int t = (warp >> 2) - 1, row = threadIdx.x & 127, wg = threadIdx.x - 128;  // wg: 0 .. 255 over both streams
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tm_s + t * kKeys + lane_base, to = tm_o + t * 128 + lane_base;
    const float scale = fabsf(a.scale_log2) > 0.f ? fabsf(a.scale_log2) : 1.f;
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale: -q with its absolute value
    const bool zero = a.scale_log2 == 0.f;                        // every score 0
    const int G = a.group;
    const uint32_t g_inv = (uint32_t)(0xFFFFFFFFu / (uint32_t)G) + 1u;  // of G > 1: r / G is the high word of r g_inv for r < 2^28
    auto token_of = [&](int r) { return G == 1 ? r : (int)__umulhi((uint32_t)r, g_inv); };
    int cnt = 0, n_o = 0, n_join = 0;
    auto all = [&] {
      const bool ok = join(joined, n_join, a.wait_limit);
      if (!ok && lane == 0) atomicOr(a.err, kErrAttend);
      return ok;
    };
    for_share(a, sh, [&](const Unit& x, int u, int s0, int s1) {
      // Q into its swizzled place (every MMA that read the previous one is done)
      constexpr int cpr = D / 8;  // 16-byte runs of a row
      const int rows32 = (x.live + 31) & ~31;  // the rows of warps that have any
      const int c = wg & (cpr - 1);
      const __half* qh = a.q + (int64_t)x.sg.row0 * a.ldq + (int64_t)x.head * G * D + 8 * c;
#pragma unroll 4
      for (int i = wg; i < rows32 * cpr; i += 256) {
        const int rr = i / cpr, r = x.r0 + rr, tok = token_of(r);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < x.n_rows && !zero) w = ldg_stream_u4(qh + (int64_t)tok * a.ldq + (r - tok * G) * D);
        w.x ^= flip, w.y ^= flip, w.z ^= flip, w.w ^= flip;
        w = in_expansion_order<KV>(w);
        *reinterpret_cast<uint4*>(q_s + (c >> 3) * C::kHalf + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = w;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mb_arrive(q_full);

      const int r = x.r0 + row;
      const int pos = x.sg.pos0 + min(r, x.n_rows - 1) / G;
      const bool busy = (warp & 3) * 32 < x.live;  // a warp without rows only keeps the barriers' count
      Reference ref(scale);
      float l = 0.f;
      for (int s = s0 + t; s < s1; s += 2, ++cnt) {
        if (!mb_wait_warp(s_full + t, cnt & 1, a.wait_limit)) {
          if (lane == 0) atomicOr(a.err, kErrAttend);
          return false;
        }
        tc_after();
        if (busy) {
          const int key = x.key0 + s * kKeys;
          const bool masked = key + kKeys - 1 > x.p_lo || (a.window && key <= x.p_hi - a.window);
          const int hi = pos - key, lo = a.window ? hi - a.window + 1 : -1;  // columns lo .. hi are seen
          auto load = [&](int c, float (&v)[32]) {
            tmem_ld32(ts + c, v);
            tmem_wait_ld();
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c + i > hi || c + i < lo) v[i] = -INFINITY;
            }
          };
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            float v[32];
            load(c, v);
            float x0 = v[0], x1 = v[1];
#pragma unroll
            for (int i = 2; i + 4 <= 32; i += 4) x0 = max3(x0, v[i], v[i + 1]), x1 = max3(x1, v[i + 2], v[i + 3]);
            top = max3(top, fmaxf(x0, x1), fmaxf(v[30], v[31]));
          }
          if (__any_sync(0xffffffffu, top > ref.m + ref.lazy)) {
            const float f = ref.raise(top, scale);
            l *= f;
            if (s > s0 + 1) {
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(to + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= f;
                tmem_st32(to + c, o);
              }
            }
          }
          const float off = ref.far ? kShift : kShift - ref.value() * scale;
          const F2 sc2 = f2(scale, scale), off2 = f2(off, off);
          F2 sum[2] = {f2(l, 0.f), f2(0.f, 0.f)};
          // P of columns c .. c + 31 goes over S's columns c / 2 .. c / 2 + 15, which are read by then
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            float v[32];
            load(c, v);
            if (ref.far) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] -= ref.value();
            }
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float e0, e1;
              unpack(fma2(f2(v[2 * i], v[2 * i + 1]), sc2, off2), e0, e1);
              const __half2 h = __floats2half2_rn(ex2(e0), ex2(e1));
              const float2 hf = __half22float2(h);
              sum[i & 1] = add2(sum[i & 1], f2(hf.x, hf.y));
              p[i] = h2_as_u32(h);
            }
            tmem_st16(ts + c / 2, p);
          }
          float a0, a1, b0, b1;
          unpack(sum[0], a0, a1);
          unpack(sum[1], b0, b1);
          l = (a0 + a1) + (b0 + b1);
          tmem_wait_st();
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mb_arrive(p_full + t);
      }
      // ---- the piece's result: stream 0's threads join the two streams, row by row
      const bool two = s1 - s0 > 1;
      if (t == 0 || two) {
        if (!mb_wait_warp(o_full + t, n_o & 1, a.wait_limit)) {
          if (lane == 0) atomicOr(a.err, kErrAttend);
          return false;
        }
        ++n_o;
      }
      tc_after();
      if (t == 1) ml_b[row] = two ? make_float2(ref.m, l) : make_float2(-INFINITY, 0.f);
      if (!all()) return false;
      const bool whole = s0 == 0 && s1 == x.n_steps;
      const int mine = 2 * (int)blockIdx.x + (u == sh.unit[blockIdx.x] ? 0 : 1);
      constexpr int kPart = (D + 2) * kRows;  // as k_attend_merge.cu reads it
      if (t == 0 && busy) {
        const float2 b = ml_b[row];
        const float mt = fmaxf(ref.m, b.x);
        const float fa = ref.m == -INFINITY ? 0.f : ex2((ref.m - mt) * scale);
        const float fb = b.x == -INFINITY ? 0.f : ex2((b.x - mt) * scale);
        const float lt = fmaf(fb, b.y, fa * l), inv = 1.0f / lt;
        const bool live = row < x.live;
        __half* dst = a.o + (int64_t)(x.sg.row0 + r / G) * a.ldo + (int64_t)(x.head * G + r % G) * D;
        float* part = a.part + (size_t)mine * kPart + row;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(to + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= fa;
          if (two) {
            float ob[32];
            tmem_ld32(to + 128 + c, ob);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(fb, ob[i], o[i]);
          }
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 32; ++i) __stcg(part + (c + i) * kRows, o[i]);
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              float y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = o[i + k] * inv;
              *reinterpret_cast<uint4*>(dst + c + i) = pack8<KV>(y);
            }
          }
        }
        if (!whole) {
          __stcg(part + D * kRows, mt);
          __stcg(part + (D + 1) * kRows, lt);
        }
      }
      tc_before();
      if (!all()) return false;  // o is read: the next piece may write it
      return true;
    });
  }
  tc_before();
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int D, int KV>
cudaError_t launch_stream_t(const Launch& L, const AttendArgs& a, const AttendShares& sh) {
  using C = Cfg<D, KV>;
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  static_assert((size_t)2 * kAttendMaxShares * kRows * (D + 2) <= kAttendPartFloats, "workspace");
  alignas(64) CUtensorMap map = {};
  cudaError_t e = KV == 0 ? pool_map(&map, a) : cudaSuccess;
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attend_stream_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(L, attend_stream_kernel<D, KV>, dim3(sh.n), dim3(C::kThreads), C::kSmem, map, a, sh);
  return e == cudaSuccess ? launch_attend_merge(L, a, sh, 1, KV == 2) : e;
}
template <int D>
cudaError_t launch_stream_kv(const Launch& L, const AttendArgs& a, const AttendShares& sh) {
  switch (a.pool.kv_dtype) {
    case 0: return launch_stream_t<D, 0>(L, a, sh);
    case 1: return launch_stream_t<D, 1>(L, a, sh);
    default: return launch_stream_t<D, 2>(L, a, sh);
  }
}

}  // namespace

cudaError_t launch_attend_stream(const Launch& L, AttendArgs& a, int n_sm) {
  if (a.n_seg < 1 || a.n_seg > MAG_MAX_BATCH) return cudaErrorInvalidValue;
  AttendShares sh;
  attend_shares(a, kRows, kKeys, n_sm, 2, 4, sh);
  return a.pool.head_dim == 64 ? launch_stream_kv<64>(L, a, sh) : launch_stream_kv<128>(L, a, sh);
}

}  // namespace mag
