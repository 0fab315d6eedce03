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

// Unit u of a row: 8 values, the units of the row's K heads first, then those of its V heads.
template <int KV>
__global__ void __launch_bounds__(kIoThreads) kv_write_kernel(const KvWriteArgs a) {
  const PoolGeom& P = a.pool;
  const int d = P.head_dim, upv = d >> 3;                 // units per vector
  const int upr = 2 * P.n_kv_heads * upv;                 // units per row
  const int row = blockIdx.x;
  const int s = seg_of_row(a.rows, row);
  const int pos = a.rows.seg[s].pos0 + row - a.rows.seg[s].row0;
  const int blk = block_of(P, a.rows.seg[s].sess, pos, a.err);
  // whole warps run to the end, so that the shuffles below have every lane (upv divides 32)
  for (int u0 = threadIdx.x & ~31; u0 < upr; u0 += kIoThreads) {
    const int u = u0 + (threadIdx.x & 31);
    const bool live = u < upr;
    const int vec = live ? u / upv : 0, e = live ? u - vec * upv : 0;
    const int part = vec >= P.n_kv_heads, head = vec - part * P.n_kv_heads;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live)
      w = ldg_stream_u4((part ? a.v : a.k) + (int64_t)row * a.ld + head * d + 8 * e);
    uint8_t* data = pool_vec(P, a.layer, blk, part, head, pos & 15);
    if (KV == 0) {
      if (live) reinterpret_cast<uint4*>(data)[e] = w;
      continue;
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
      uint32_t c[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int q = 0;
        if (sc != 0.0f) q = max(-127, min(127, (int)rintf(__fdiv_rn(x[i], sc))));
        c[i >> 2] |= (uint32_t)(q & 255) << (8 * (i & 3));
      }
      if (live) {
        reinterpret_cast<uint2*>(data)[e] = make_uint2(c[0], c[1]);
        if (e == 0) *reinterpret_cast<__half*>(pool_vec(P, a.layer, blk, part + 2, head, pos & 15)) = s16;
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
      uint32_t c = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int q = 0;
        if (sc != 0.0f) q = max(0, min(15, (int)rintf(__fdiv_rn(__fsub_rn(x[i], mn), sc))));
        c |= (uint32_t)q << (4 * i);
      }
      if (live) {
        reinterpret_cast<uint32_t*>(data)[e] = c;
        if ((e & 3) == 0)
          reinterpret_cast<__half2*>(pool_vec(P, a.layer, blk, part + 2, head, pos & 15))[e >> 2] =
              __halves2half2(s16, m16);
      }
    }
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
      for (int i = 0; i < 4; ++i) {  // codes (i, i + 4) as fp16 1024 + q
        const uint32_t h = ((c >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
        r[i] = h2_as_u32(__hfma2(__hsub2(u32_as_h2(h), u32_as_h2(0x64006400u)), sc, mn));
      }
      o = make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                     __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
    }
    const int64_t row = sg.row0 + pos - sg.pos0;
    *reinterpret_cast<uint4*>(out + row * a.ld + head * d + 8 * e) = o;
  }
}

}  // namespace

cudaError_t launch_kv_write(const Launch& L, const KvWriteArgs& a) {
  const int n = a.rows.n_rows;
  if (n < 1 || a.rows.n_seg < 1 || a.rows.n_seg > MAG_MAX_BATCH) return cudaErrorInvalidValue;
  if (a.pool.kv_dtype == 0) kv_write_kernel<0><<<n, kIoThreads, 0, L.stream>>>(a);
  else if (a.pool.kv_dtype == 1) kv_write_kernel<1><<<n, kIoThreads, 0, L.stream>>>(a);
  else kv_write_kernel<2><<<n, kIoThreads, 0, L.stream>>>(a);
  if (L.counter) ++*L.counter;
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const Launch& L, const KvReadArgs& a, int n_layers) {
  if (a.n_blocks < 1 || n_layers < 1 || n_layers > 65535 || a.rows.n_seg < 1 || a.rows.n_seg > MAG_MAX_BATCH)
    return cudaErrorInvalidValue;
  const dim3 grid(a.n_blocks, 2, n_layers);
  if (a.pool.kv_dtype == 0) kv_read_kernel<0><<<grid, kIoThreads, 0, L.stream>>>(a);
  else if (a.pool.kv_dtype == 1) kv_read_kernel<1><<<grid, kIoThreads, 0, L.stream>>>(a);
  else kv_read_kernel<2><<<grid, kIoThreads, 0, L.stream>>>(a);
  if (L.counter) ++*L.counter;
  return cudaGetLastError();
}

}  // namespace mag
