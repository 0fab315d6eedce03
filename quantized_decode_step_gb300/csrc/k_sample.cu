// Sampling of the next token from rows of logits: temperature, top-k, top-p and min-p, with given random numbers.
//
// The tokens of a row stand in order (logit falling, equal logits by index rising); w_i = exp((l_i - max) / T) and
// every cut keeps a prefix of that order: top-k its first k tokens, top-p the shortest prefix of those whose w add
// up to top_p of theirs, min-p the tokens with w >= min_p. The token is the first of the shortest prefix whose
// running sum of w passes u times the prefix's sum.
//
// A row is never sorted: each of the (up to) three places in that order, the k-th token, the end of top-p and the
// token itself, is found by a radix descent over the logits as ordered integers, on histograms of counts and of
// weights. The weights are integers, w in units of 2^-40 to within 2^-33 of their value (a table of 2^(-j/256) and a
// polynomial for the rest, the exponent in two fp32 terms), so that their sums are exact in 64 bits: no
// order of atomics changes a result, prefixes found on different histograms agree to the last unit, and a token
// differs from that of real arithmetic only where u falls within about 1e-10 of a border.
//
// What bounds it: one read of the logits (a row of 128,256 in fp16 is 0.04 us of HBM time), so in practice the
// latency of the passes. A cluster of blocks shares a row: each keeps its slice of the row in shared memory as ordered
// integers, later passes read only those, and histograms are added up through distributed shared memory. As
// many blocks to a row as the row count leaves SMs for.
#include <cooperative_groups.h>

#include <algorithm>

#include "kernels.h"

namespace mag {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kTopBits = 11, kTopBins = 1 << kTopBits;  // first digit of the descent
constexpr int kMaxBins = 128;                           // bins of a later digit
constexpr int kMaxCluster = 8;
constexpr size_t kKeyBytes = 150 * 1024;                // most bytes of a slice
constexpr int kOneShift = 40;                           // w = 1 is 2^40

// 2^(-j / 256) in units of 2^-40, j = 0 .. 255.
struct ExpTable {
  unsigned long long v[256];
};
constexpr ExpTable make_exp_table() {
  ExpTable t{};
  for (int j = 0; j < 256; ++j) {
    // e^(-j ln 2 / 256) by its series: the argument is below ln 2, 24 terms leave less than 2^-60
    const double x = -0.693147180559945309417232121458 * j / 256.0;
    double term = 1.0, sum = 0.0;
    for (int k = 0; k < 24; ++k) {
      sum += term;
      term *= x / (k + 1);
    }
    t.v[j] = (unsigned long long)(sum * 1099511627776.0 + 0.5);
  }
  return t;
}
__device__ constexpr ExpTable kExpTable = make_exp_table();

template <typename T>
struct Keys;
// fp16: the ordered key is 16 bits, fp32: 32. Key 0 stands for a token that may not be drawn (below every number).
template <>
struct Keys<__half> {
  using Key = uint16_t;
  static constexpr int kBits = 16, kDigits = 1, kDigitBits = 5;
  static constexpr int kPer16 = 8;
  __device__ static Key of(__half h) {
    const float f = __half2float(h);
    if (!(f > -INFINITY)) return 0;  // NaN and -inf
    const uint16_t b = f == 0.f ? 0 : __half_as_ushort(h);  // -0 is 0
    return (b & 0x8000u) ? (uint16_t)~b : (uint16_t)(b | 0x8000u);
  }
  __device__ static float value(uint32_t k) {
    return __half2float(__ushort_as_half((k & 0x8000u) ? (uint16_t)(k & 0x7FFFu) : (uint16_t)~k));
  }
};
template <>
struct Keys<float> {
  using Key = uint32_t;
  static constexpr int kBits = 32, kDigits = 3, kDigitBits = 7;
  static constexpr int kPer16 = 4;
  __device__ static Key of(float f) {
    if (!(f > -INFINITY)) return 0;
    const uint32_t b = f == 0.f ? 0u : __float_as_uint(f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  }
  __device__ static float value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
  }
};

// exp((x - max) / T) in units of 2^-40; kh + kl = log2(e) / T.
struct Weight {
  float mx, kh, kl;
  const unsigned long long* table;
  __device__ unsigned long long operator()(float x) const {
    // max - x as s + e, exactly; times log2(e) / T as th + tl
    const float s = __fsub_rn(mx, x);
    const float bb = __fsub_rn(s, mx);
    const float e = __fsub_rn(__fsub_rn(mx, __fsub_rn(s, bb)), __fadd_rn(x, bb));
    const float th = s * kh;
    // below 2^-48, less than half a unit; infinite logits (s is NaN between them) have all the weight
    if (!(th < 48.0f)) return x == mx ? 1ull << kOneShift : 0ull;
    const float tl = fmaf(s, kh, -th) + fmaf(s, kl, e * kh);
    const float i = rintf(th * 256.0f);
    const float r = -((th - i * 0.00390625f) + tl);  // 2^-(th + tl) = 2^(-i / 256) 2^r
    const float c = r * fmaf(r, fmaf(r, fmaf(r, 9.6181291e-3f, 5.5504109e-2f), 0.24022651f), 0.69314718f);
    const int ii = (int)i;
    const unsigned long long w0 = table[ii & 255];
    const float f0 = (float)(uint32_t)(w0 >> 9) * 512.0f;
    const unsigned long long w = w0 + (long long)__float2int_rn(f0 * c);
    const int sh = ii >> 8;
    return sh ? (w + (1ull << (sh - 1))) >> sh : w;
  }
};

struct Place {            // a place in the falling order: the tie of key `key` with number `tie` (from 1)
  uint32_t key;
  uint32_t above_n, tie_n;  // tokens above the key, tokens of the key
  unsigned long long above_w;
  uint32_t tie;
};

template <typename T>
struct SampleSmem {
  unsigned long long w1[kTopBins], w1c[kTopBins];   // this block's histogram, the row's
  uint32_t c1[kTopBins], c1c[kTopBins];
  unsigned long long wd[3][Keys<T>::kDigits][kMaxBins];
  uint32_t cd[3][Keys<T>::kDigits][kMaxBins];
  unsigned long long table[256];
  unsigned long long scan_w[kThreads / 32];
  uint32_t scan_c[kThreads / 32];
  unsigned long long best;       // (key, ~index) of this block's largest
  unsigned long long min_sum;    // sum of the weights at or above min-p's
  uint32_t min_key;
  // results of the descents
  uint32_t bin;
  uint32_t above_n;
  unsigned long long above_w;
  uint32_t found;
  unsigned long long comb_w[kMaxBins];
  uint32_t comb_c[kMaxBins];
};

__device__ __forceinline__ unsigned long long warp_incl(unsigned long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ uint32_t warp_incl(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

template <typename T>
class Row {
 public:
  using KT = Keys<T>;
  using Key = typename KT::Key;
  __device__ Row(SampleSmem<T>& sm, Key* keys, int n, Weight w, cg::cluster_group cl)
      : sm_(sm), keys_(keys), n_(n), w_(w), cl_(cl) {}

  // f(key, index in the slice) over the slice, whole 16-byte runs of the keys per thread.
  template <typename F>
  __device__ void each(F f) const {
    constexpr int P = KT::kPer16;
    for (int c = threadIdx.x; c * P < n_; c += kThreads) {
      Key k[P];
      *reinterpret_cast<uint4*>(k) = reinterpret_cast<const uint4*>(keys_)[c];
#pragma unroll
      for (int i = 0; i < P; ++i) f((uint32_t)k[i], c * P + i);
    }
  }

  // The first place whose running count (by_count) or weight reaches target; false if the row has less.
  // `slot`: which of the three digit histograms to use.
  __device__ bool find(bool by_count, unsigned long long target, int slot, Place& out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int per = kTopBins / kThreads;
    // the first digit: thread tid owns the bins tid * per .. from the top
    unsigned long long w[per], ws = 0;
    uint32_t c[per], cs = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const int b = kTopBins - 1 - (tid * per + i);
      w[i] = sm_.w1c[b], c[i] = sm_.c1c[b];
      ws += w[i], cs += c[i];
    }
    unsigned long long wi = warp_incl(ws, lane);
    uint32_t ci = warp_incl(cs, lane);
    if (tid == 0) sm_.found = 0;
    if (lane == 31) sm_.scan_w[warp] = wi, sm_.scan_c[warp] = ci;
    __syncthreads();
    unsigned long long wb = wi - ws;
    uint32_t cb = ci - cs;
    for (int i = 0; i < warp; ++i) wb += sm_.scan_w[i], cb += sm_.scan_c[i];
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const unsigned long long before = by_count ? cb : wb, here = by_count ? c[i] : w[i];
      if (before < target && target <= before + here) {
        sm_.bin = kTopBins - 1 - (tid * per + i);
        sm_.above_n = cb, sm_.above_w = wb;
        sm_.found = 1;
      }
      wb += w[i], cb += c[i];
    }
    __syncthreads();
    if (!sm_.found) return false;  // the same in every block of the cluster
    uint32_t prefix = sm_.bin;
    int shift = KT::kBits - kTopBits;
#pragma unroll 1
    for (int dg = 0; dg < KT::kDigits; ++dg) {
      constexpr int bins = 1 << KT::kDigitBits;
      const bool last = dg == KT::kDigits - 1;
      const int low = shift - KT::kDigitBits;
      each([&](uint32_t k, int) {
        if ((k >> shift) == prefix) {
          const uint32_t b = (k >> low) & (bins - 1);
          atomicAdd(&sm_.cd[slot][dg][b], 1u);
          if (!last) {
            const unsigned long long x = w_(KT::value(k));
            if (x) atomicAdd(&sm_.wd[slot][dg][b], x);
          }
        }
      });
      cl_.sync();
      const int nb = cl_.num_blocks();
      if (tid < bins) {
        uint32_t cc = 0;
        unsigned long long ww = 0;
        for (int r = 0; r < nb; ++r) {
          cc += *cl_.map_shared_rank(&sm_.cd[slot][dg][tid], r);
          if (!last) ww += *cl_.map_shared_rank(&sm_.wd[slot][dg][tid], r);
        }
        if (last && cc) ww = cc * w_(KT::value((prefix << KT::kDigitBits) | tid));
        sm_.comb_c[tid] = cc, sm_.comb_w[tid] = ww;
      }
      __syncthreads();
      if (warp == 0) {
        constexpr int pl = bins / 32;
        unsigned long long lw = 0;
        uint32_t lc = 0;
#pragma unroll
        for (int i = 0; i < pl; ++i) {
          const int b = bins - 1 - (lane * pl + i);
          lw += sm_.comb_w[b], lc += sm_.comb_c[b];
        }
        unsigned long long bw = sm_.above_w + warp_incl(lw, lane) - lw;
        uint32_t bc = sm_.above_n + warp_incl(lc, lane) - lc;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < pl; ++i) {
          const int b = bins - 1 - (lane * pl + i);
          const unsigned long long before = by_count ? bc : bw, here = by_count ? sm_.comb_c[b] : sm_.comb_w[b];
          if (before < target && target <= before + here) sm_.bin = b, sm_.above_n = bc, sm_.above_w = bw;
          bw += sm_.comb_w[b], bc += sm_.comb_c[b];
        }
      }
      __syncthreads();
      prefix = (prefix << KT::kDigitBits) | sm_.bin;
      shift = low;
    }
    out.key = prefix;
    out.above_n = sm_.above_n, out.above_w = sm_.above_w;
    out.tie_n = sm_.comb_c[sm_.bin];
    if (by_count) {
      out.tie = (uint32_t)(target - out.above_n);
    } else {
      const unsigned long long w1 = w_(KT::value(prefix));
      out.tie = (uint32_t)((target - out.above_w + w1 - 1) / w1);
    }
    __syncthreads();
    return true;
  }

  // Index in the slice of the slice's `tie`-th (from 1) token of key `key`, or -1: one thread gets it.
  __device__ int locate(uint32_t key, uint32_t tie) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n_ + kThreads - 1) / kThreads, i0 = min(n_, tid * per), i1 = min(n_, i0 + per);
    uint32_t mine = 0;
    for (int i = i0; i < i1; ++i) mine += keys_[i] == key;
    const uint32_t incl = warp_incl(mine, lane);
    if (lane == 31) sm_.scan_c[warp] = incl;
    __syncthreads();
    uint32_t before = incl - mine;
    for (int i = 0; i < warp; ++i) before += sm_.scan_c[i];
    if (before < tie && tie <= before + mine)
      for (int i = i0; i < i1; ++i)
        if (keys_[i] == key && ++before == tie) return i;
    return -1;
  }

 private:
  SampleSmem<T>& sm_;
  Key* keys_;
  int n_;
  Weight w_;
  cg::cluster_group cl_;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs a) {
  using KT = Keys<T>;
  using Key = typename KT::Key;
  constexpr int P = KT::kPer16;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SampleSmem<T>& sm = *reinterpret_cast<SampleSmem<T>*>(smem_raw);
  Key* keys = reinterpret_cast<Key*>(smem_raw + (sizeof(SampleSmem<T>) + 15) / 16 * 16);
  cg::cluster_group cl = cg::this_cluster();
  const int nb = cl.num_blocks(), rank = cl.block_rank();
  const int row = blockIdx.x / nb, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // the slice: runs of P tokens, the row's cut into nb parts
  const T* x = reinterpret_cast<const T*>(a.logits) + (int64_t)row * a.ld;
  const int runs = (a.vocab + P - 1) / P, per = (runs + nb - 1) / nb;
  const int v0 = min(a.vocab, rank * per * P), v1 = min(a.vocab, v0 + per * P), n = v1 - v0;
  const uint32_t* bits = a.allowed ? a.allowed + (int64_t)row * ((a.vocab + 31) / 32) : nullptr;
  const bool wide = (reinterpret_cast<uintptr_t>(x + v0) & 15) == 0;

  for (int i = tid; i < kTopBins; i += kThreads) sm.w1[i] = 0, sm.c1[i] = 0;
  for (int i = tid; i < 3 * KT::kDigits * kMaxBins; i += kThreads)
    (&sm.wd[0][0][0])[i] = 0, (&sm.cd[0][0][0])[i] = 0;
  if (tid < 256) sm.table[tid] = kExpTable.v[tid];
  unsigned long long best = 0;
  for (int c = tid; c * P < n; c += kThreads) {
    T v[P];
    const int i0 = v0 + c * P, live = min(P, v1 - i0);
    if (wide && live == P) {
      *reinterpret_cast<uint4*>(v) = ldg_stream_u4(x + i0);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < live) v[i] = x[i0 + i];
    }
    // the run's bits lie in one word (P divides 32, v0 is a multiple of P)
    const uint32_t ok = bits ? bits[i0 >> 5] >> (i0 & 31) : 0xffffffffu;
    Key k[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      k[i] = i < live && ((ok >> i) & 1) ? KT::of(v[i]) : (Key)0;
      const unsigned long long cand = ((unsigned long long)k[i] << 32) | (uint32_t)~(i0 + i);
      best = cand > best ? cand : best;
    }
    *reinterpret_cast<uint4*>(keys + c * P) = *reinterpret_cast<uint4*>(k);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const unsigned long long u = __shfl_xor_sync(0xffffffffu, best, o);
    best = u > best ? u : best;
  }
  if (lane == 0) sm.scan_w[warp] = best;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kThreads / 32; ++i) best = sm.scan_w[i] > best ? sm.scan_w[i] : best;
    sm.best = best;
    sm.min_sum = 0;
    sm.min_key = 0xffffffffu;
  }
  cl.sync();
  best = 0;
  for (int r = 0; r < nb; ++r) {
    const unsigned long long u = *cl.map_shared_rank(&sm.best, r);
    best = u > best ? u : best;
  }
  const uint32_t top = (uint32_t)(best >> 32);
  const float temp = a.temperature ? a.temperature[row] : 1.0f;
  const double kd = 1.4426950408889634073599 / (double)temp;
  const float kh = (float)kd;
  // no token may be drawn, or the largest one is taken (temperature not above zero, or too small to divide by)
  if (top == 0 || !(temp > 0.f) || isinf(kh)) {
    if (rank == 0 && tid == 0) {
      a.token[row] = top == 0 ? -1 : (int32_t)~(uint32_t)best;
      if (a.prob) a.prob[row] = top == 0 ? __int_as_float(0x7fc00000) : 1.0f;
    }
    cl.sync();  // no block leaves while another reads its shared memory
    return;
  }
  const Weight w{KT::value(top), kh, (float)(kd - (double)kh), sm.table};
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.0f, min_p = a.min_p ? a.min_p[row] : 0.0f;
  const bool use_k = top_k > 0 && top_k < a.vocab, use_p = top_p < 1.0f, use_m = min_p > 0.0f;
  const double one = (double)(1ull << kOneShift);
  // the least weight that min-p keeps (above one: only the first token)
  const unsigned long long least =
      use_m ? (min_p > 1.0f ? (1ull << kOneShift) + 1 : (unsigned long long)ceil((double)min_p * one)) : 0ull;

  Row<T> rw(sm, keys, n, w, cl);
  unsigned long long msum = 0;
  uint32_t mkey = 0xffffffffu;
  rw.each([&](uint32_t k, int) {
    if (!k) return;
    const uint32_t b = k >> (KT::kBits - kTopBits);
    const unsigned long long v = w(KT::value(k));
    if (v) atomicAdd(&sm.w1[b], v);
    if (use_k) atomicAdd(&sm.c1[b], 1u);
    if (use_m && v >= least) {
      msum += v;
      mkey = min(mkey, k);
    }
  });
  if (use_m) {
    atomicAdd(&sm.min_sum, msum);
    atomicMin(&sm.min_key, mkey);
  }
  cl.sync();
  // the row's histogram: block r adds up its share of the bins, then everyone takes all of them
  {
    const int share = kTopBins / nb;
    for (int i = tid; i < share; i += kThreads) {
      const int b = rank * share + i;
      unsigned long long ww = 0;
      uint32_t cc = 0;
      for (int r = 0; r < nb; ++r) {
        ww += *cl.map_shared_rank(&sm.w1[b], r);
        cc += *cl.map_shared_rank(&sm.c1[b], r);
      }
      sm.w1c[b] = ww, sm.c1c[b] = cc;
    }
    cl.sync();
    for (int i = tid; i < kTopBins; i += kThreads) {
      const int owner = i / share;
      if (owner != rank) {
        sm.w1c[i] = *cl.map_shared_rank(&sm.w1c[i], owner);
        sm.c1c[i] = *cl.map_shared_rank(&sm.c1c[i], owner);
      }
    }
  }
  unsigned long long m_sum = 0;
  uint32_t m_key = 0xffffffffu;
  if (use_m)
    for (int r = 0; r < nb; ++r) {
      m_sum += *cl.map_shared_rank(&sm.min_sum, r);
      m_key = min(m_key, *cl.map_shared_rank(&sm.min_key, r));
    }
  __syncthreads();

  // the kept prefix: its last key, how many of that key's tokens, its sum
  uint32_t end_key = 0, end_tie = 0xffffffffu;
  unsigned long long total;
  Place at;
  {
    unsigned long long s = 0;
    for (int i = lane; i < kTopBins; i += 32) s += sm.w1c[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    total = s;
  }
  if (use_k && rw.find(true, (unsigned long long)top_k, 0, at)) {
    end_key = at.key, end_tie = at.tie;
    total = at.above_w + at.tie * w(KT::value(at.key));
  }
  if (use_p) {
    const double t = ceil((double)top_p * (double)total);
    const unsigned long long target = t >= 1.0 ? min((unsigned long long)t, total) : 1ull;
    if (rw.find(false, target, 1, at)) {
      end_key = at.key, end_tie = at.tie;
      total = at.above_w + at.tie * w(KT::value(at.key));
    }
  }
  if (use_m) {
    if (m_key == 0xffffffffu) {  // min-p above one
      total = 1ull << kOneShift;
    } else if (m_key > end_key) {
      total = m_sum;
    }
  }
  const float u = a.uniform[row];
  const double tu = floor((double)u * (double)total);
  const unsigned long long target = tu >= 0.0 ? min((unsigned long long)tu + 1, total) : 1ull;
  if (rw.find(false, target, 2, at)) {
    // the block that holds the tie: the blocks' counts of this key are in their last digit's histograms
    const int b = at.key & ((1 << KT::kDigitBits) - 1);
    uint32_t before = 0, mine = 0;
    for (int r = 0; r <= rank; ++r) {
      mine = *cl.map_shared_rank(&sm.cd[2][KT::kDigits - 1][b], r);
      if (r < rank) before += mine;
    }
    if (before < at.tie && at.tie <= before + mine) {
      const int i = rw.locate(at.key, at.tie - before);
      if (i >= 0) {
        a.token[row] = v0 + i;
        if (a.prob) a.prob[row] = (float)((double)w(KT::value(at.key)) / (double)total);
      }
    }
  }
  cl.sync();
}

template <typename T>
cudaError_t launch_sample_t(cudaStream_t s, const SampleArgs& a) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const size_t head = (sizeof(SampleSmem<T>) + 15) / 16 * 16;
  auto slice = [&](int nb) {
    constexpr int P = Keys<T>::kPer16;
    const int runs = (a.vocab + P - 1) / P;
    return (size_t)((runs + nb - 1) / nb) * 16;
  };
  // as many blocks to a row as there are SMs for, each with at least a run for every second thread
  int nb = 1;
  while (nb < kMaxCluster && (slice(nb) > kKeyBytes || ((int64_t)a.rows * nb * 2 <= n_sm && slice(nb) > kThreads * 8)))
    nb *= 2;
  if (slice(nb) > kKeyBytes) return cudaErrorInvalidValue;
  const size_t smem = head + slice(nb);
  e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * nb));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nb;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
}

}  // namespace

int64_t sample_max_vocab(bool f32) { return (int64_t)kMaxCluster * (kKeyBytes / (f32 ? 4 : 2)); }

cudaError_t launch_sample(cudaStream_t s, const SampleArgs& a) {
  if (a.rows < 1 || a.vocab < 1 || a.vocab > sample_max_vocab(a.f32)) return cudaErrorInvalidValue;
  return a.f32 ? launch_sample_t<float>(s, a) : launch_sample_t<__half>(s, a);
}

}  // namespace mag
