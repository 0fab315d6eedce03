// Attention of the newest tokens of several sessions over one layer's block pool, for many rows: tcgen05.
//
//   o_t = sum_j softmax_j(scale q_t . k_j) v_j   over the keys j <= p_t, and j > p_t - window if there is one,
//
// the G query heads of a KV head and the tokens of a session packed into rows t G + g, so one read of a key serves
// them all. What bounds it is the tensor core: 4 d flops a row and key, 2 x 128 x 128 x d a tile for Q K^T and as many for
// P V, against 32 KB of K and V from L2.
//
// A unit is 256 rows (two tiles of 128) of one session and KV head over their keys in steps of 128. One block per
// SM takes an equal share of all units' steps, in order, so that every SM works to the end whatever the causal
// triangle leaves of the units; a unit cut by a share's end leaves (m, l, o) in the workspace, whose parts a second
// kernel (k_attend_merge.cu) puts together.
//
// Roles: one warp loads K and V of a step into a ring of swizzled tiles (FP16 by TMA, a 16-token pool block and 64
// dimensions a copy; INT8 and INT4 as raw bytes that four warps expand to the fp16 values the pool reads
// back as); one thread issues the MMAs; a warpgroup per row tile takes S from tensor memory, one row a
// thread, and leaves P there in fp16 over S's columns, where the second MMA reads it as its A operand, with V as it
// lies (its rows are the contraction: an MN-major B operand). While one tile's softmax runs, the tensor core
// has the other tile's P V and its next Q K^T.
//
// Softmax: as in the few-row kernel, base 2 with a maximum that is raised only when a score passes it by more
// than 2^8 (the rescaling of o in tensor memory is then rare; scores far from zero: Reference) and p scaled by 2^7 before
// its rounding to fp16. The sum adds p in fp32 before the rounding, so o is off by up to 2^-11 of itself where all roundings go
// one way: the rounded p, which the other kernels add, cost 1,107 us for 1,058 on 4,096 tokens and 19,431 keys (with
// mixed-precision adds; 1,143 widened first), since the softmax is not wholly hidden here.
//
// Every wait is bounded; a role whose wait gives up sets a bit in the error word and leaves, after its own copies
// and MMAs in flight.
#include <algorithm>

#include "attend_tc.cuh"

namespace mag {

namespace {

using namespace tc;

// ---------------------------------------------------------------- shapes
template <int D, int KV>
struct Cfg {
  static constexpr int kTile = kKeys * D * 2;          // one K or V tile, or a Q tile, in fp16
  static constexpr int kHalf = kKeys * 128;            // its 64-dimension halves
  static constexpr int kStages = D == 128 ? (KV == 0 ? 5 : 4) : 8;
  static constexpr int kRowB = KV == 0 ? 2 * D : (KV == 1 ? D : D / 2), kMetaB = KV == 0 ? 0 : (KV == 1 ? 2 : D / 8);
  static constexpr int kRawData = kKeys * kRowB, kRawMeta = kKeys * kMetaB;
  static constexpr int kRaw = KV == 0 ? 0 : 2;         // slots of raw bytes
  static constexpr int kRawBytes = KV == 0 ? 0 : kRawData + kRawMeta;
  static constexpr int kThreads = KV == 0 ? 384 : 512;
  // registers: 384 x 168 or 512 x 128 at launch. The softmax wants them (256 tokens on 20,000 INT4 keys: 96 us so, 100 at
  // 184 and 72, 133 at 168 and 88); FP16 is the same from 200 to 216.
  static constexpr int kRegsSoftmax = 200, kRegsOther = KV == 0 ? 104 : 56;
  static_assert(256 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= kThreads * (KV == 0 ? 168 : 128), "registers");
  static constexpr int kBars = 2 * kStages + 2 * kRaw + 9;
  static constexpr int kSmem = 2 * kTile + kStages * kTile + kRaw * kRawBytes + kBars * 8 + 64 + 1024;
};

struct Unit {
  AttendSeg sg;
  int head, r0, n_rows;   // first packed row, rows of the session
  int p_lo, p_hi;         // positions of the unit's first and last token
  int key0, n_steps;      // first key (a pool block's first), steps
};

// Unit u: (session, head, tile pair), the pair fastest.
__device__ __forceinline__ Unit unit_at(const AttendArgs& a, int u) {
  Unit x;
  int si = 0;
  for (int i = 1; i < a.n_seg; ++i)
    if (u >= a.seg[i].unit0) si = i;
  x.sg = a.seg[si];
  const int v = u - x.sg.unit0;
  x.head = v / x.sg.n_tiles;
  x.r0 = (v - x.head * x.sg.n_tiles) * 2 * kRows;
  x.n_rows = x.sg.n_tok * a.group;
  x.n_steps = attend_unit_steps(x.sg.pos0, x.n_rows, a.group, a.window, x.r0, 2 * kRows, kKeys, x.p_lo, x.p_hi, x.key0);
  return x;
}

// f(unit, index, first step, end step) for every piece of this block's share.
template <typename F>
__device__ __forceinline__ void for_share(const AttendArgs& a, const AttendShares& sh, F f) {
  int u = sh.unit[blockIdx.x], s = sh.step[blockIdx.x];
  const int ue = sh.unit[blockIdx.x + 1], se = sh.step[blockIdx.x + 1];
  while (u < ue || (u == ue && s < se)) {
    const Unit x = unit_at(a, u);
    const int e = u == ue ? se : x.n_steps;
    if (!f(x, u, s, e)) return;
    ++u;
    s = 0;
  }
}

// 8 stored values (INT8: words c0 and c1, offset by 128; INT4: word c0) as fp16 in order.
template <int KV>
__device__ __forceinline__ uint4 expand8(uint32_t c0, uint32_t c1, uint32_t meta) {
  uint32_t r[4];
  const __half2 s = __low2half2(u32_as_h2(meta));
  if constexpr (KV == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = __byte_perm((i < 2 ? c0 : c1) ^ 0x80808080u, 0x64646464u, (i & 1) ? 0x4342 : 0x4140);
      r[i] = h2_as_u32(__hmul2(__hsub2(u32_as_h2(h), u32_as_h2(0x64806480u)), s));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  } else {
    const __half2 m = __high2half2(u32_as_h2(meta));
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = h2_as_u32(__hfma2(u4_pair(c0, i), s, m));
    return make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                      __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
  }
}

template <int D, int KV>
__global__ void __launch_bounds__(Cfg<D, KV>::kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ AttendArgs a,
                     const __grid_constant__ AttendShares sh) {
  using C = Cfg<D, KV>;
  constexpr int ST = C::kStages, RAW = C::kRaw;
  constexpr uint32_t kIdescQK = (1u << 4) | ((uint32_t)(kKeys >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
  constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;                         // [2][128 rows x D]
  uint8_t* ring = smem + 2 * C::kTile;         // [ST][128 keys x D]
  uint8_t* raw = ring + ST * C::kTile;         // [RAW] stored bytes: data, then scales
  uint64_t* full = reinterpret_cast<uint64_t*>(raw + RAW * C::kRawBytes);
  uint64_t* empty = full + ST;
  uint64_t* raw_full = empty + ST;
  uint64_t* raw_empty = raw_full + RAW;
  uint64_t* q_full = raw_empty + RAW;  // [2]: Q of the tile is in shared memory
  uint64_t* s_full = q_full + 2;   // [2]: S of the tile is in tensor memory (and o holds every earlier step)
  uint64_t* p_full = s_full + 2;   // [2]: P is
  uint64_t* o_full = p_full + 2;   // [2]: o is final
  uint64_t* mma_done = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PoolGeom& P = a.pool;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mb_init(full + i, KV == 0 ? 1 : 4);
      mb_init(empty + i, 1);
    }
    for (int i = 0; i < RAW; ++i) {
      mb_init(raw_full + i, 1);
      mb_init(raw_empty + i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mb_init(q_full + i, 4);
      mb_init(s_full + i, 1);
      mb_init(p_full + i, 4);
      mb_init(o_full + i, 1);
    }
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
  const uint32_t tm_s = tmem, tm_o = tmem + 2 * kKeys;  // S (and P) of tile t at + 128 t, o of tile t at + 128 t

  pdl_trigger();  // the merge kernel may be put in place; it waits for this grid's end
  if (warp < 4) {
    regs_dec<C::kRegsOther>();
    if (warp == 0) {
      // ---- loader: K and V of every step, in the order the MMAs use them
      const int32_t* table = nullptr;
      const uint8_t* layer_base = P.base + (int64_t)a.layer * P.pool_blocks * P.block_bytes;
      const int64_t data_part = (int64_t)P.n_kv_heads * 16 * C::kRowB, meta_part = (int64_t)P.n_kv_heads * 16 * C::kMetaB;
      int g = 0;
      for_share(a, sh, [&](const Unit& x, int, int s0, int s1) {
        table = P.tables + (int64_t)x.sg.sess * P.table_stride;
        const int len = x.sg.pos0 + x.sg.n_tok, n_blk = (len + 15) >> 4;
        int ids = 0;
        for (int s = s0; s < s1; ++s) {
          const int key = x.key0 + s * kKeys, b0 = key >> 4;
          if (((s - s0) & 3) == 0) {  // the ids of four steps, one a lane
            const int b = b0 + lane;
            ids = b < n_blk ? checked_block(table[b], (int)P.pool_blocks, a.err) : 0;
          }
          const int nb = min(8, n_blk - b0);                  // pool blocks of this step
          const int nv = min(8, (len - key) >> 4);            // of them, whole ones
          const int my = __shfl_sync(0xffffffffu, ids, ((s - s0) & 3) * 8 + (lane & 7));
          for (int part = 0; part < 2; ++part, ++g) {
            if constexpr (KV == 0) {
              const int st = g % ST;
              if (g >= ST && !mb_wait_warp(empty + st, ((g / ST) - 1) & 1, a.wait_limit)) {
                if (lane == 0) atomicOr(a.err, kErrAttend);
                return false;
              }
              const uint32_t dst = su32(ring + st * C::kTile);
              int n_tma = nb;
              if (part == 1 && nv < 8) {
                // the step that holds the session's end: value rows past it are zeros (a slot there may hold anything,
                // and 0 times it must be 0), the block it lies in is copied row by row
                n_tma = nv;
                const int y0 = nv * 16;
                for (int i = lane; i < (kKeys - y0) * (D / 8); i += 32) {  // a multiple of 32
                  const int row = y0 + i / (D / 8), c = i % (D / 8);
                  uint4 w = make_uint4(0, 0, 0, 0);
                  const int b = __shfl_sync(0xffffffffu, ids, ((s - s0) & 3) * 8 + (row >> 4));
                  if (key + row < len)
                    w = *reinterpret_cast<const uint4*>(layer_base + (int64_t)b * P.block_bytes + data_part +
                                                        ((int64_t)x.head * 16 + (row & 15)) * C::kRowB + 16 * c);
                  *reinterpret_cast<uint4*>(ring + st * C::kTile + (c >> 3) * C::kHalf + row * 128 +
                                            (((c & 7) ^ (row & 7)) << 4)) = w;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
              }
              if (lane == 0) mb_expect(full + st, (uint32_t)n_tma * 16 * D * 2);
              __syncwarp();
              const int blk = lane & 7, half = lane >> 3;
              if (blk < n_tma && half < D / 64)
                tma_3d(dst + half * C::kHalf + blk * 2048, &map, half * 64, (part * P.n_kv_heads + x.head) * 16, my,
                       full + st);
            } else {
              const int r = g % RAW;
              if (g >= RAW && !mb_wait_warp(raw_empty + r, ((g / RAW) - 1) & 1, a.wait_limit)) {
                if (lane == 0) atomicOr(a.err, kErrAttend);
                return false;
              }
              const uint32_t dst = su32(raw + r * C::kRawBytes);
              if (lane == 0) mb_expect(raw_full + r, (uint32_t)nb * 16 * (C::kRowB + C::kMetaB));
              __syncwarp();
              const int blk = lane & 7;
              const uint8_t* base = layer_base + (int64_t)my * P.block_bytes;
              if (lane < nb)
                bulk_g2s(dst + blk * 16 * C::kRowB, base + part * data_part + (int64_t)x.head * 16 * C::kRowB,
                         16 * C::kRowB, raw_full + r);
              else if (lane >= 8 && lane < 8 + nb)
                bulk_g2s(dst + C::kRawData + blk * 16 * C::kMetaB,
                         base + 2 * data_part + part * meta_part + (int64_t)x.head * 16 * C::kMetaB, 16 * C::kMetaB,
                         raw_full + r);
            }
          }
        }
        return true;
      });
      // leave no copy in flight, also when a consumer gave up and will not wait for it
      if constexpr (KV == 0) {
        for (int f = max(0, g - ST); f < g; ++f) mb_wait(full + f % ST, (f / ST) & 1);
      } else {
        for (int f = max(0, g - RAW); f < g; ++f) mb_wait(raw_full + f % RAW, (f / RAW) & 1);
      }
    } else if (warp == 1 && lane == 0) {
      // ---- MMA issuer
      int g = 0, pieces[2] = {0, 0}, cnt[2] = {0, 0};
      const uint32_t q_a = su32(q_s), ring_a = su32(ring);
      auto qk = [&](int t, int st) {
        const uint64_t qd = smem_desc(q_a + t * C::kTile, 16), kd = smem_desc(ring_a + st * C::kTile, 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = (uint64_t)((k >> 2) * C::kHalf + (k & 3) * 32) >> 4;
          mma_ss(tm_s + t * kKeys, qd + off, kd + off, kIdescQK, k != 0);
        }
        mma_commit(s_full + t);
      };
      for_share(a, sh, [&](const Unit& x, int, int s0, int s1) {
        const int nt = x.n_rows - x.r0 > kRows ? 2 : 1, n = s1 - s0;
        bool ok = mb_wait(full + g % ST, (g / ST) & 1, a.wait_limit);
        for (int t = 0; t < nt && ok; ++t) ok = mb_wait(q_full + t, pieces[t] & 1, a.wait_limit);
        if (ok) {
          tc_after();
          for (int t = 0; t < nt; ++t) qk(t, g % ST);
          mma_commit(empty + g % ST);
          for (int j = 0; j < n && ok; ++j) {
            const int gv = g + 1 + 2 * j, sv = gv % ST, sk = (gv + 1) % ST;
            const bool next = j + 1 < n;
            ok = mb_wait(full + sv, (gv / ST) & 1, a.wait_limit);
            for (int t = 0; t < nt && ok; ++t) {
              ok = mb_wait(p_full + t, (cnt[t] + j) & 1, a.wait_limit);
              if (!ok) break;
              tc_after();
              const uint64_t vd = smem_desc(ring_a + sv * C::kTile, C::kHalf);
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                mma_ts(tm_o + t * 128, tm_s + t * kKeys + k * 8, vd + ((uint64_t)(k * 2048) >> 4), kIdescPV,
                       (j | k) != 0);
              if (next) {
                if (t == 0) {
                  ok = mb_wait(full + sk, ((gv + 1) / ST) & 1, a.wait_limit);
                  if (!ok) break;
                  tc_after();
                }
                qk(t, sk);
              } else {
                mma_commit(o_full + t);
              }
            }
            if (!ok) break;
            mma_commit(empty + sv);
            if (next) mma_commit(empty + sk);
          }
        }
        if (!ok) {
          atomicOr(a.err, kErrAttend);
          return false;
        }
        g += 2 * n;
        for (int t = 0; t < nt; ++t) ++pieces[t], cnt[t] += n;
        return true;
      });
      // every MMA has completed before the block frees its tensor memory
      mma_commit(mma_done);
      mb_wait(mma_done, 0);
    }
  } else if (KV != 0 && warp >= 12) {
    // ---- expansion of INT8 / INT4 tiles, 16 stored bytes of a row a thread at a time
    regs_dec<C::kRegsOther>();
    if constexpr (KV != 0) {
      const int w = warp - 12;
      // 8 lanes side by side have 8 rows, and of each the run that makes the banks that they read differ; the runs that
      // they write differ then too (64 INT4 values: two by two the same)
      constexpr int kRuns = C::kRowB / 16;
      const int b1 = (lane >> 1) & 1, b2 = (lane >> 2) & 1;
      const int turn = C::kRowB == 128 ? lane & 7 : (C::kRowB == 32 ? b2 : (KV == 1 ? 2 * b1 + (b2 ^ b1) : 2 * b2 + b1));
      int g = 0;
      for_share(a, sh, [&](const Unit& x, int, int s0, int s1) {
        const int len = x.sg.pos0 + x.sg.n_tok;
        for (int s = s0; s < s1; ++s) {
          const int live = len - (x.key0 + s * kKeys);  // rows that hold tokens
          for (int part = 0; part < 2; ++part, ++g) {
            const int r = g % RAW, st = g % ST;
            if (!mb_wait_warp(raw_full + r, (g / RAW) & 1, a.wait_limit) ||
                (g >= ST && !mb_wait_warp(empty + st, ((g / ST) - 1) & 1, a.wait_limit))) {
              if (lane == 0) atomicOr(a.err, kErrAttend);
              return false;
            }
            const uint8_t* src = raw + r * C::kRawBytes;
            uint8_t* dst = ring + st * C::kTile;
#pragma unroll 1
            for (int i = 0; i < kKeys * kRuns / 128; ++i) {
              const int item = (i * 4 + w) * 32 + lane, row = (item & 7) | (item / (8 * kRuns) << 3);
              const int run = ((item >> 3) % kRuns) ^ turn;
              uint4 c = make_uint4(0, 0, 0, 0);
              uint32_t meta = 0;
              if (row < live) {
                c = *reinterpret_cast<const uint4*>(src + row * C::kRowB + 16 * run);
                const uint8_t* mp = src + C::kRawData + row * C::kMetaB;
                meta = KV == 1 ? *reinterpret_cast<const uint16_t*>(mp) : reinterpret_cast<const uint32_t*>(mp)[run];
              }
              const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
              constexpr int NE = KV == 1 ? 2 : 4;  // fp16 runs of a stored one
#pragma unroll
              for (int e = 0; e < NE; ++e) {
                const int cc = NE * run + e;
                const uint4 v = KV == 1 ? expand8<KV>(cw[2 * (e & 1)], cw[2 * (e & 1) + 1], meta) : expand8<KV>(cw[e], 0, meta);
                *reinterpret_cast<uint4*>(dst + (cc >> 3) * C::kHalf + row * 128 + (((cc & 7) ^ (row & 7)) << 4)) = v;
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              mb_arrive(raw_empty + r);
              mb_arrive(full + st);
            }
          }
        }
        return true;
      });
    }
  } else {
    // ---- softmax of row tile t, one row a thread
    regs_inc<C::kRegsSoftmax>();
    const int t = (warp >> 2) - 1, row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tm_s + t * kKeys + lane_base, to = tm_o + t * 128 + lane_base;
    const float scale = fabsf(a.scale_log2) > 0.f ? fabsf(a.scale_log2) : 1.f;
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale: -q with its absolute value
    const bool zero = a.scale_log2 == 0.f;                        // every score 0
    const int G = a.group;
    const uint32_t g_inv = (uint32_t)(0xFFFFFFFFu / (uint32_t)G) + 1u;  // of G > 1: r / G is the high word of r g_inv for r < 2^28
    auto token_of = [&](int r) { return G == 1 ? r : (int)__umulhi((uint32_t)r, g_inv); };
    int cnt = 0, n_o = 0;
    for_share(a, sh, [&](const Unit& x, int u, int s0, int s1) {
      // Q of the tile into its swizzled place (every MMA that read the previous one is done)
      if (x.n_rows - x.r0 <= t * kRows) return true;  // no such tile
      {
        uint8_t* qt = q_s + t * C::kTile;
        constexpr int cpr = D / 8;  // 16-byte runs of a row
        // a thread has one run of every 128 / cpr-th row; all its loads first
        const int c = threadIdx.x & (cpr - 1), rr0 = (threadIdx.x & 127) / cpr;
        const __half* qh = a.q + (int64_t)x.sg.row0 * a.ldq + (int64_t)x.head * G * D + 8 * c;
        uint4 w[cpr];
#pragma unroll
        for (int i = 0; i < cpr; ++i) {
          const int r = x.r0 + t * kRows + rr0 + i * (128 / cpr), tok = token_of(r);
          w[i] = make_uint4(0, 0, 0, 0);
          if (r < x.n_rows && !zero) w[i] = ldg_stream_u4(qh + (int64_t)tok * a.ldq + (r - tok * G) * D);
        }
#pragma unroll
        for (int i = 0; i < cpr; ++i) {
          const int rr = rr0 + i * (128 / cpr);
          *reinterpret_cast<uint4*>(qt + (c >> 3) * C::kHalf + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) =
              make_uint4(w[i].x ^ flip, w[i].y ^ flip, w[i].z ^ flip, w[i].w ^ flip);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) mb_arrive(q_full + t);

      const int r = x.r0 + t * kRows + row;
      const int pos = x.sg.pos0 + min(r, x.n_rows - 1) / G;
      // positions of the tile's first and last token: which steps need a mask
      const int t_lo = x.sg.pos0 + (x.r0 + t * kRows) / G;
      const int t_hi = x.sg.pos0 + (min(x.r0 + t * kRows + kRows, x.n_rows) - 1) / G;
      Reference ref(scale);
      float l = 0.f;
      for (int s = s0; s < s1; ++s, ++cnt) {
        if (!mb_wait_warp(s_full + t, cnt & 1, a.wait_limit)) {
          if (lane == 0) atomicOr(a.err, kErrAttend);
          return false;
        }
        tc_after();
        float v[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(ts + c, v + c);
        tmem_wait_ld();
        const int key = x.key0 + s * kKeys;
        if (key + kKeys - 1 > t_lo || (a.window && key <= t_hi - a.window)) {
          const int hi = pos - key, lo = a.window ? hi - a.window + 1 : -1;  // columns lo .. hi are seen
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (c > hi || c < lo) v[c] = -INFINITY;
        }
        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int c = 4; c + 8 <= kKeys; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], v[c + i], v[c + 4 + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], v[kKeys - 4 + i]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (__any_sync(0xffffffffu, top > ref.m + ref.lazy)) {
          const float f = ref.raise(top, scale);
          l *= f;
          if (s > s0) {
#pragma unroll
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
        if (ref.far) {
          // from S once more, 32 columns at a time: as a branch over v it cost every step 4% (4,096 tokens on 19,431)
          const float m = ref.value();
          const int hi = pos - (x.key0 + s * kKeys), lo = a.window ? hi - a.window + 1 : -1;
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 32) {
            float w[32];
            tmem_ld32(ts + c, w);
            tmem_wait_ld();
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const bool in0 = c + 2 * i <= hi && c + 2 * i >= lo, in1 = c + 2 * i + 1 <= hi && c + 2 * i + 1 >= lo;
              const float e0 = in0 ? ex2(fmaf(w[2 * i] - m, scale, kShift)) : 0.f;
              const float e1 = in1 ? ex2(fmaf(w[2 * i + 1] - m, scale, kShift)) : 0.f;
              l += e0 + e1;
              p[i] = h2_as_u32(__floats2half2_rn(e0, e1));
            }
            tmem_st16(ts + c / 2, p);
          }
        } else {
          const float off = kShift - ref.value() * scale;
          const F2 sc2 = f2(scale, scale), off2 = f2(off, off);
          F2 sum[2] = {f2(l, 0.f), f2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float e0, e1;
              unpack(fma2(f2(v[c + 2 * i], v[c + 2 * i + 1]), sc2, off2), e0, e1);
              e0 = ex2(e0), e1 = ex2(e1);
              sum[i & 1] = add2(sum[i & 1], f2(e0, e1));
              p[i] = h2_as_u32(__floats2half2_rn(e0, e1));
            }
            tmem_st16(ts + c / 2, p);
          }
          float a0, a1, b0, b1;
          unpack(sum[0], a0, a1);
          unpack(sum[1], b0, b1);
          l = (a0 + a1) + (b0 + b1);
        }
        tmem_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mb_arrive(p_full + t);
      }
      // ---- the piece's result
      if (!mb_wait_warp(o_full + t, n_o & 1, a.wait_limit)) {
        if (lane == 0) atomicOr(a.err, kErrAttend);
        return false;
      }
      ++n_o;
      tc_after();
      const bool live = r < x.n_rows;
      __half* dst = a.o + (int64_t)(x.sg.row0 + r / G) * a.ldo + (int64_t)(x.head * G + r % G) * D;
      auto store = [&](int c, const float* o, float inv) {
        if (!live) return;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint4 w;
          w.x = h2_as_u32(__floats2half2_rn(o[i] * inv, o[i + 1] * inv));
          w.y = h2_as_u32(__floats2half2_rn(o[i + 2] * inv, o[i + 3] * inv));
          w.z = h2_as_u32(__floats2half2_rn(o[i + 4] * inv, o[i + 5] * inv));
          w.w = h2_as_u32(__floats2half2_rn(o[i + 6] * inv, o[i + 7] * inv));
          *reinterpret_cast<uint4*>(dst + c + i) = w;
        }
      };
      if (s0 == 0 && s1 == x.n_steps) {
        const float inv = 1.0f / l;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(to + c, o);
          tmem_wait_ld();
          store(c, o, inv);
        }
        return true;
      }
      // a cut unit: this block's part, column by column ([2 per block][tile][D + 2][128])
      constexpr int kPart = (D + 2) * kRows;
      const int mine = 2 * (int)blockIdx.x + (u == sh.unit[blockIdx.x] ? 0 : 1);
      float* part = a.part + (int64_t)(2 * mine + t) * kPart + row;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(to + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) __stcg(part + (c + i) * kRows, o[i]);
      }
      __stcg(part + D * kRows, ref.m);
      __stcg(part + (D + 1) * kRows, l);
      return true;
    });
  }
  tc_before();
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int D, int KV>
cudaError_t launch_tc_t(const Launch& L, const AttendArgs& a, const AttendShares& sh) {
  using C = Cfg<D, KV>;
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  alignas(64) CUtensorMap map = {};
  cudaError_t e = KV == 0 ? pool_map(&map, a) : cudaSuccess;
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attend_tc_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(L, attend_tc_kernel<D, KV>, dim3(sh.n), dim3(C::kThreads), C::kSmem, map, a, sh);
  return e == cudaSuccess ? launch_attend_merge(L, a, sh, 2, false) : e;
}
template <int D>
cudaError_t launch_tc_kv(const Launch& L, const AttendArgs& a, const AttendShares& sh) {
  switch (a.pool.kv_dtype) {
    case 0: return launch_tc_t<D, 0>(L, a, sh);
    case 1: return launch_tc_t<D, 1>(L, a, sh);
    default: return launch_tc_t<D, 2>(L, a, sh);
  }
}

}  // namespace

cudaError_t launch_attend_tc(const Launch& L, AttendArgs& a, int n_sm) {
  if (a.n_seg < 1 || a.n_seg > MAG_MAX_BATCH) return cudaErrorInvalidValue;
  // every block at least two steps: a merge costs about as much
  AttendShares sh;
  attend_shares(a, 2 * kRows, kKeys, n_sm, 2, 4, sh);
  return a.pool.head_dim == 64 ? launch_tc_kv<64>(L, a, sh) : launch_tc_kv<128>(L, a, sh);
}

}  // namespace mag
