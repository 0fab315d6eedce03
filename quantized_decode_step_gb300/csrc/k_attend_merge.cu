// The parts that the tcgen05 attention kernels leave of units whose keys went to several blocks, put together:
//
//   o = sum_b 2^(scale (m_b - m)) o_b / sum_b 2^(scale (m_b - m)) l_b,   m = max_b m_b,   in the blocks' order.
//
// A part is [D values, m, l][128 rows] in fp32, column by column, as the kernels' threads, one row each, write it.
// What bounds it: reading the parts from L2 (64 KB a tile and part), so it is a kernel of its own: the last block of a unit to
// arrive took 6.4 us over two parts of 256 rows, and four times as long over 19 of 128. A warp has 32 rows, one a lane,
// and 8 columns. Launched as a dependent of the attention kernel, so that its launch is not waited for.
#include "kernels.h"

namespace mag {

namespace {

constexpr int kWarps = 8;

template <int D, bool PERM>
__global__ void __launch_bounds__(kWarps * 32) attend_merge_kernel(const __grid_constant__ AttendArgs a,
                                                                   const __grid_constant__ AttendCuts cuts, int tiles) {
  constexpr int CW = 8, CG = D / (CW * kWarps);  // columns of a warp, blocks over the columns
  pdl_wait();
  const int lane = threadIdx.x & 31, c0 = ((blockIdx.x % CG) * kWarps + (threadIdx.x >> 5)) * CW;
  const int b = blockIdx.x / CG, cut = b / (4 * tiles), tile = b / 4 % tiles, row = (b & 3) * 32 + lane;
  int si = 0;
  const int u = cuts.unit[cut];
  for (int i = 1; i < a.n_seg; ++i)
    if (u >= a.seg[i].unit0) si = i;
  const AttendSeg sg = a.seg[si];
  const int head = (u - sg.unit0) / sg.n_tiles, pair = u - sg.unit0 - head * sg.n_tiles;
  const int r = (pair * tiles + tile) * 128 + row;  // packed row of the session
  if (r - lane >= sg.n_tok * a.group) return;
  const int b0 = cuts.first[cut], b1 = cuts.last[cut], slot0 = cuts.slot[cut];
  constexpr int kPart = (D + 2) * 128;
  const float scale = fabsf(a.scale_log2) > 0.f ? fabsf(a.scale_log2) : 1.f;  // as the kernels take it
  auto part_of = [&](int b) {
    return a.part + (int64_t)((b == b0 ? slot0 : 2 * b) * tiles + tile) * kPart + row;
  };
  // eight parts at a time, all their loads before the first use: the latency of L2 is what a group costs
  constexpr int GP = 8;
  float m = -INFINITY, l = 0.f, o[CW];
#pragma unroll
  for (int i = 0; i < CW; ++i) o[i] = 0.f;
  for (int b = b0; b <= b1; b += GP) {
    float mb[GP], lb[GP], v[GP][CW];
#pragma unroll
    for (int k = 0; k < GP; ++k) {
      mb[k] = -INFINITY, lb[k] = 0.f;
#pragma unroll
      for (int i = 0; i < CW; ++i) v[k][i] = 0.f;
      if (b + k <= b1) {
        const float* p = part_of(b + k);
        mb[k] = __ldcg(p + D * 128);
        lb[k] = __ldcg(p + (D + 1) * 128);
#pragma unroll
        for (int i = 0; i < CW; ++i) v[k][i] = __ldcg(p + (c0 + i) * 128);
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < GP; ++k) mn = fmaxf(mn, mb[k]);
    const float f0 = m == -INFINITY ? 0.f : exp2f((m - mn) * scale);
    m = mn;
    l *= f0;
#pragma unroll
    for (int i = 0; i < CW; ++i) o[i] *= f0;
#pragma unroll
    for (int k = 0; k < GP; ++k) {
      if (mb[k] == -INFINITY) continue;  // nothing there (a part of masked keys, or past the last)
      const float f = exp2f((mb[k] - m) * scale);
      l = fmaf(f, lb[k], l);
#pragma unroll
      for (int i = 0; i < CW; ++i) o[i] = fmaf(f, v[k][i], o[i]);
    }
  }
  if (r >= sg.n_tok * a.group) return;
  const float inv = 1.0f / l;
  __half* dst = a.o + (int64_t)(sg.row0 + r / a.group) * a.ldo + (int64_t)(head * a.group + r % a.group) * D + c0;
  float x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[PERM ? (k & 1) * 4 + (k >> 1) : k] = o[k] * inv;
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(h2_as_u32(__floats2half2_rn(x[0], x[1])), h2_as_u32(__floats2half2_rn(x[2], x[3])),
                 h2_as_u32(__floats2half2_rn(x[4], x[5])), h2_as_u32(__floats2half2_rn(x[6], x[7])));
}

template <int D, bool PERM>
cudaError_t launch_merge_t(const Launch& L, const AttendArgs& a, const AttendCuts& cuts, int tiles) {
  return launch_kernel(Launch{L.stream, true, L.counter}, attend_merge_kernel<D, PERM>, dim3(cuts.n * tiles * 4 * (D / 64)),
                       dim3(kWarps * 32), 0, a, cuts, tiles);
}

}  // namespace

cudaError_t launch_attend_merge(const Launch& L, const AttendArgs& a, const AttendShares& sh, int tiles, bool perm) {
  AttendCuts cuts = {};
  for (int b = 1; b < sh.n; ++b) {
    if (sh.step[b] == 0) continue;
    if (cuts.n && cuts.unit[cuts.n - 1] == sh.unit[b]) {
      cuts.last[cuts.n - 1] = b;
      continue;
    }
    cuts.unit[cuts.n] = sh.unit[b];
    cuts.first[cuts.n] = b - 1;
    cuts.last[cuts.n] = b;
    cuts.slot[cuts.n] = 2 * (b - 1) + (sh.unit[b - 1] == sh.unit[b] ? 0 : 1);
    ++cuts.n;
  }
  if (!cuts.n) return cudaSuccess;
  if (a.pool.head_dim == 64)
    return perm ? launch_merge_t<64, true>(L, a, cuts, tiles) : launch_merge_t<64, false>(L, a, cuts, tiles);
  return perm ? launch_merge_t<128, true>(L, a, cuts, tiles) : launch_merge_t<128, false>(L, a, cuts, tiles);
}

}  // namespace mag
