// One layer's cache traffic as calls of their own: new keys and values of several sessions quantised into the
// block pool as they are written, and stored tokens read back as fp16.
//
// Formats ("5. Core modules" 5.4: FP16 / INT8 / INT4 KV), per (token, head) vector of d values:
//   FP16  the values;
//   INT8  s = fp16(max|x| / 127), q = clamp(rint(x / s), -127, 127)   (s = 0: q = 0);
//   INT4  per 32 values m = fp16(min), s = fp16((max - min) / 15), q = clamp(rint((x - m) / s), 0, 15).
// The decisions are taken in fp32 with IEEE division and round-half-even, as by the bulk store, so the stored
// bytes are the same. A stored value reads back as fp16(s q) or fp16(s q + m): one fp16 multiply or
// multiply-add, so rounded once from the exact product (the codes are exact in fp16).
//
// Both directions are bound by memory: a thread owns 8 values (16 bytes of fp16), a quarter of an INT4 group, so a
// vector is d / 8 neighbouring lanes, its maximum (or its groups' minima and maxima) a few shuffles, and every
// fp16 access a whole 16-byte run.
#include "kernels.h"

namespace mag {

namespace {

constexpr int kIoThreads = 256;

__device__ __forceinline__ int seg_of_row(const KvRows& r, int row) {
  int s = 0;
  for (int i = 1; i < r.n_seg; ++i)
    if (row >= r.seg[i].row0) s = i;
  return s;
}

// The pool place of one (row, K/V, head): block id checked against the pool.
__device__ __forceinline__ int block_of(const PoolGeom& P, int sess, int pos, uint32_t* err) {
  return checked_block(P.tables[(int64_t)sess * P.table_stride + (pos >> 4)], (int)P.pool_blocks, err);
}

// rint(x / s) of 8 values as clamp(.., lo, hi), as IEEE division and round-half-even decide it, without a division for
// most: q = rint(x / s) from the reciprocal, and the remainder x - q s, which fp32 holds exactly, says how far the
// quotient lies from halfway between two codes. Within 2^-17 of that (the reciprocal's quotient is off by at most 2^-18
// for codes up to 15; up to 127, quotients of fp16 numbers are halfway or at least 2^-12 off) the division decides.
// A scale below fp16's normal numbers is rounded coarsely: only then can a quotient pass the codes' range.
__device__ __forceinline__ void codes8(const float (&x)[8], float s, int lo, int hi, int (&q)[8]) {
  const float inv = s != 0.f ? 1.0f / s : 0.f;  // 0: every code 0
  float close = INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float m = fmaf(x[i], inv, 12582912.0f), r = fmaf(-(m - 12582912.0f), s, x[i]);
    q[i] = __float_as_int(m) - 0x4B400000;
    close = fminf(close, fabsf(fmaf(2.0f, fabsf(r), -s)));
  }
  if (s != 0.f && (close <= s * 1.52587890625e-5f || s < 6.103515625e-5f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = max(lo, min(hi, (int)rintf(__fdiv_rn(x[i], s))));
  }
}

// The stored form of 8 values of one vector, by the d / 8 neighbouring lanes that have it (e: which of them).
template <int KV>
__device__ __forceinline__ void store8(const PoolGeom& P, int layer, int blk, int part, int head, int slot, int e, int upv,
                                       const uint4& w, bool live) {
  uint8_t* data = pool_vec(P, layer, blk, part, head, slot);
  if (KV == 0) {
    if (live) reinterpret_cast<uint4*>(data)[e] = w;
    return;
  }
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(u32_as_h2(ww[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  if (KV == 1) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
    for (int o = upv >> 1; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const __half s16 = __float2half_rn(__fdiv_rn(amax, 127.0f));
    const float sc = __half2float(s16);
    int q[8];
    codes8(x, sc, -127, 127, q);
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i >> 2] |= (uint32_t)(q[i] & 255) << (8 * (i & 3));
    if (live) {
      reinterpret_cast<uint2*>(data)[e] = make_uint2(c[0], c[1]);
      if (e == 0) *reinterpret_cast<__half*>(pool_vec(P, layer, blk, part + 2, head, slot)) = s16;
    }
  } else {
    // minimum and maximum of the group's 4 lanes; of equal minima the first in index order (the sign of zero)
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      if (x[i] < lo) lo = x[i];
      if (x[i] > hi) hi = x[i];
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float l2 = __shfl_xor_sync(0xffffffffu, lo, o), h2 = __shfl_xor_sync(0xffffffffu, hi, o);
      const bool first = (threadIdx.x & o) == 0;
      if (l2 < lo || (l2 == lo && !first)) lo = l2;
      if (h2 > hi) hi = h2;
    }
    const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const __half m16 = __float2half_rn(lo);
    const float sc = __half2float(s16), mn = __half2float(m16);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fsub_rn(x[i], mn);
    int q[8];
    codes8(x, sc, 0, 15, q);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) c |= (uint32_t)q[i] << (4 * i);
    if (live) {
      reinterpret_cast<uint32_t*>(data)[e] = c;
      if ((e & 3) == 0)
        reinterpret_cast<__half2*>(pool_vec(P, layer, blk, part + 2, head, slot))[e >> 2] = __halves2half2(s16, m16);
    }
  }
}

// A block has NR neighbouring rows; unit u of a row: 8 values, the units of its K heads first, then those of its V
// heads. A thread loads its unit of all NR rows before it stores the first.
template <int KV, int NR>
__global__ void __launch_bounds__(kIoThreads) kv_write_kernel(const __grid_constant__ KvWriteArgs a) {
  const PoolGeom& P = a.pool;
  const int d = P.head_dim, upv = d >> 3;                 // units per vector
  const int upr = 2 * P.n_kv_heads * upv;                 // units per row
  const int row0 = blockIdx.x * NR;
  __shared__ int s_blk[NR], s_slot[NR];
  if (threadIdx.x < NR && row0 + threadIdx.x < a.rows.n_rows) {
    const int row = row0 + threadIdx.x, s = seg_of_row(a.rows, row);
    const int pos = a.rows.seg[s].pos0 + row - a.rows.seg[s].row0;
    s_blk[threadIdx.x] = block_of(P, a.rows.seg[s].sess, pos, a.err);
    s_slot[threadIdx.x] = pos & 15;
  }
  const int nr = min(NR, a.rows.n_rows - row0);
  int part, head, e;
  bool live;
  uint4 w[NR];
  auto load = [&](int u0) {  // of this lane's unit in the warp's units u0 .. u0 + 31
    const int u = u0 + (threadIdx.x & 31);
    live = u < upr;
    const int vec = live ? u / upv : 0;
    e = live ? u - vec * upv : 0;
    part = vec >= P.n_kv_heads, head = vec - part * P.n_kv_heads;
    const __half* src = (part ? a.v : a.k) + (int64_t)row0 * a.ld + head * d + 8 * e;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      w[r] = make_uint4(0, 0, 0, 0);
      if (live && r < nr) w[r] = ldg_stream_u4(src + r * a.ld);
    }
  };
  // whole warps run to the end, so that store8's shuffles have every lane (upv divides 32)
  int u0 = threadIdx.x & ~31;
  if (u0 < upr) load(u0);
  __syncthreads();  // the rows' places
  while (u0 < upr) {
#pragma unroll
    for (int r = 0; r < NR; ++r)
      if (r < nr) store8<KV>(P, a.layer, s_blk[r], part, head, s_slot[r], e, upv, w[r], live);
    u0 += kIoThreads;
    if (u0 < upr) load(u0);
  }
}

// One block per 16-token pool block (blockIdx.x), K or V (y) and layer (z): its stored bytes are one run.
template <int KV>
__global__ void __launch_bounds__(kIoThreads) kv_read_kernel(const KvReadArgs a) {
  const PoolGeom& P = a.pool;
  const int d = P.head_dim, upv = d >> 3, part = blockIdx.y, layer = a.layer + blockIdx.z;
  // this block's session and table index
  int s = 0;
  for (int i = 1; i < a.rows.n_seg; ++i)
    if ((int)blockIdx.x >= a.blk0[i]) s = i;
  const KvSeg sg = a.rows.seg[s];
  const int t16 = (sg.pos0 >> 4) + blockIdx.x - a.blk0[s];
  const int p0 = max(sg.pos0, t16 * 16), p1 = min(sg.pos0 + sg.n_tok, t16 * 16 + 16);
  const int phys = block_of(P, sg.sess, t16 * 16, a.err);
  __half* out = (part ? a.v : a.k) + (int64_t)blockIdx.z * a.layer_stride;
  const int n_units = P.n_kv_heads * 16 * upv;
#pragma unroll 4
  for (int u = threadIdx.x; u < n_units; u += kIoThreads) {
    const int vec = u / upv, e = u - vec * upv, head = vec >> 4, slot = vec & 15;
    const int pos = t16 * 16 + slot;
    if (pos < p0 || pos >= p1) continue;
    const uint8_t* data = pool_vec(P, layer, phys, part, head, slot);
    uint4 o;
    if (KV == 0) {
      o = ldg_stream_u4(data + 16 * e);
    } else if (KV == 1) {
      const uint2 c = ldg_stream_u2(data + 8 * e);
      const __half2 sc = __half2half2(*reinterpret_cast<const __half*>(pool_vec(P, layer, phys, part + 2, head, slot)));
      const uint32_t cw[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // bytes (2i, 2i + 1), offset by 128, as fp16 1024 + byte; minus 1152 is the code, exactly
        const uint32_t h = __byte_perm(cw[i >> 1], 0x64646464u, (i & 1) ? 0x4342 : 0x4140);
        r[i] = h2_as_u32(__hmul2(__hsub2(u32_as_h2(h), u32_as_h2(0x64806480u)), sc));
      }
      o = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
      const uint32_t c = ldg_nc_u32(data + 4 * e);
      const __half2 sm =
          reinterpret_cast<const __half2*>(pool_vec(P, layer, phys, part + 2, head, slot))[e >> 2];
      const __half2 sc = __low2half2(sm), mn = __high2half2(sm);
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = h2_as_u32(__hfma2(u4_pair(c, i), sc, mn));
      o = make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                     __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
    }
    const int64_t row = sg.row0 + pos - sg.pos0;
    *reinterpret_cast<uint4*>(out + row * a.ld + head * d + 8 * e) = o;
  }
}

}  // namespace

template <int KV>
static cudaError_t launch_write_t(const Launch& L, const KvWriteArgs& a) {
  // one row a block leaves no load waiting for another row's; of many rows, four a block keep more bytes in flight
  // (7,000 rows of 8 heads, d 128, INT4, with their read-back: 28.3 us for 32.4; 16 rows of INT8: 9.6 us for 7.7)
  const int n = a.rows.n_rows;
  return n <= 512 ? launch_kernel(L, kv_write_kernel<KV, 1>, dim3(n), dim3(kIoThreads), 0, a)
                  : launch_kernel(L, kv_write_kernel<KV, 4>, dim3((n + 3) / 4), dim3(kIoThreads), 0, a);
}

cudaError_t launch_kv_write(const Launch& L, const KvWriteArgs& a) {
  const int n = a.rows.n_rows;
  if (n < 1 || a.rows.n_seg < 1 || a.rows.n_seg > MAG_MAX_BATCH) return cudaErrorInvalidValue;
  return a.pool.kv_dtype == 0 ? launch_write_t<0>(L, a) : (a.pool.kv_dtype == 1 ? launch_write_t<1>(L, a) : launch_write_t<2>(L, a));
}

cudaError_t launch_kv_read(const Launch& L, const KvReadArgs& a, int n_layers) {
  if (a.n_blocks < 1 || n_layers < 1 || n_layers > 65535 || a.rows.n_seg < 1 || a.rows.n_seg > MAG_MAX_BATCH)
    return cudaErrorInvalidValue;
  const dim3 grid(a.n_blocks, 2, n_layers);
  auto kernel = a.pool.kv_dtype == 0 ? kv_read_kernel<0> : (a.pool.kv_dtype == 1 ? kv_read_kernel<1> : kv_read_kernel<2>);
  return launch_kernel(L, kernel, grid, dim3(kIoThreads), 0, a);
}

}  // namespace mag
