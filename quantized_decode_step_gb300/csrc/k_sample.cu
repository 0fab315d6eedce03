// Sampling of the next token from rows of logits: temperature, top-k, top-p and min-p, with given random numbers.
//
// The tokens of a row stand in order (logit falling, equal logits by index rising); w_i = exp((l_i - max) / T) and
// every cut keeps a prefix of that order: top-k its first k tokens, top-p the shortest prefix of those whose w add
// up to top_p of theirs, min-p the tokens with w >= min_p. The token is the first of the shortest prefix whose
// running sum of w passes u times the prefix's sum.
//
// A row is never sorted. Its tokens fall into 2,048 bins by t = (max - l) log2(e) / T, so the bins stand in the
// tokens' order, each with its count and its sum of w. Every place looked for (the k-th token, the end of
// top-p, the token itself) lies in one bin, found on the bins' running sums; only that bin's tokens (the
// first k and their last bin, with top-k) are gathered and sorted. Where they are more than kCap, mostly
// equal logits, a radix descent over the logits as ordered integers finds the place instead.
//
// The weights are integers, w in units of 2^-40 to within 2^-30 of their value (a table of 2^(-j/256), a cubic for the
// rest, t in two fp32 terms), so that their sums are exact in 64 bits: no order of atomics changes a result,
// sums over different sets of the same tokens agree to the last unit, and a token differs from that of real
// arithmetic only where u falls within about 1e-9 / sqrt(tokens) of a border.
//
// What bounds it: the logits are read once (256 rows of 128,256 in fp16: 10 us of HBM time), so with few rows the
// latency of the passes between cluster barriers, with many the about 40 instructions a token of the weights. A
// cluster of blocks shares a row, each with its slice of the row in shared memory; as many blocks to a row as the
// row count leaves SMs for.
#include <cooperative_groups.h>

#include <algorithm>

#include "kernels.h"

namespace mag {

namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 2048;
constexpr int kCap = 1024;             // most tokens gathered and sorted
constexpr int kMaxCluster = 8;
constexpr size_t kKeyBytes = 144 * 1024;  // most bytes of a slice
constexpr int kOneShift = 40;          // w = 1 is 2^40
constexpr float kMaxT = 41.0f;         // tokens of t >= 41 weigh less than half a unit
constexpr int kDigits = 4, kDigitBins = 256;

// 2^(-j / 256) in units of 2^-31, j = 0 .. 255, and the same as a float.
struct ExpTable {
  uint32_t v[256];
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
    t.v[j] = (uint32_t)(sum * 2147483648.0 + 0.5);
  }
  return t;
}
__device__ constexpr ExpTable kExpTable = make_exp_table();

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }

// Ordered key of a number that is not NaN (-0 as 0); larger logits have larger keys.
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// exp((x - max) / T) in units of 2^-40; kh + kl = log2(e) / T.
struct Weight {
  float mx, kh, kl;
  const uint2* table;
  // t to fp32: what decides a token's bin. NaN for a token that cannot be drawn, and between infinite logits.
  __device__ __forceinline__ float t(float x) const { return __fmul_rn(__fsub_rn(mx, x), kh); }
  __device__ __forceinline__ unsigned long long operator()(float x) const {
    // max - x as s + e, exactly; times log2(e) / T as th + tl
    const float s = __fsub_rn(mx, x);
    const float bb = __fsub_rn(s, mx);
    const float e = __fsub_rn(__fsub_rn(mx, __fsub_rn(s, bb)), __fadd_rn(x, bb));
    const float th = __fmul_rn(s, kh);
    if (!(th < kMaxT)) return x == mx ? 1ull << kOneShift : 0ull;
    const float tl = fmaf(s, kh, -th) + fmaf(s, kl, e * kh);
    // th = i / 256 + ..: i and, below, the integer part of a product by adding 1.5 2^23
    const float im = fmaf(th, 256.0f, 12582912.0f);
    const int i = __float_as_int(im) - 0x4B400000;
    const float r = -(fmaf(im - 12582912.0f, -0.00390625f, th) + tl);  // 2^-(th + tl) = 2^(-i / 256) 2^r
    const float c = r * fmaf(r, fmaf(r, 5.5504109e-2f, 0.24022651f), 0.69314718f);
    const uint2 w0 = table[i & 255];
    const uint32_t m = w0.x + (__float_as_int(fmaf(__uint_as_float(w0.y), c, 12582912.0f)) - 0x4B400000);
    const int sh = i >> 8;
    return sh < 10 ? (unsigned long long)m << (9 - sh) : (unsigned long long)(((m >> (sh - 10)) + 1) >> 1);
  }
};

// A histogram of weights: 64-bit adds to shared memory are compare-and-swap loops (59 clocks a warp on logits' bins
// against 22 for the loop around them, 1,700 on one bin), 32-bit adds are not (22 and 34). So a weight goes in as three
// limbs of 14, 14 and 13 bits: a slice has fewer than 2^17 tokens, so a limb's sum stays below 2^31.
template <int N>
struct Limbs {
  uint32_t v[3][N];
  __device__ __forceinline__ void add(int b, unsigned long long w) {
    atomicAdd(&v[0][b], (uint32_t)w & 0x3FFFu);
    if (w >> 14) atomicAdd(&v[1][b], (uint32_t)(w >> 14) & 0x3FFFu);
    if (w >> 28) atomicAdd(&v[2][b], (uint32_t)(w >> 28));
  }
};

typedef unsigned long long u64;

struct Place {      // a place in the falling order: tie number `tie` (from 1) of key `key`
  u64 above_w;      // weight of the keys above
  uint32_t key, tie;
  int32_t index;    // the token, -1 where only key and tie are known
};

template <int NB>
struct SampleSmem {
  Limbs<kBins> w1;   // this block's histogram; later two lists of gathered tokens
  uint32_t c1[kBins];
  union {            // zero up to here at the start
    struct {         // combine: the row's bins that this block adds up
      u64 own_w[NB == 1 ? 1 : kBins / NB];
      uint32_t own_n[NB == 1 ? 1 : kBins / NB];
    };
    struct {         // gather: tokens of the row, (key, ~index), then sorted, and their running weights
      u64 cand[kCap];
      u64 cum[kCap];
    };
    struct {         // descend: a histogram per digit
      Limbs<kDigitBins> wd[kDigits];
      uint32_t cd[kDigits][kDigitBins];
    };
  };
  u64 wa[kBins + 1];           // weight above bin b, tokens above bin b
  uint32_t na[kBins + 1];
  uint2 table[256];
  u64 red_w[32];
  uint32_t red_c[32], red_d[32];
  float2 ext;                  // this block's largest and least logit
  u64 min_sum;                 // weight of the tokens that min-p keeps, and the least key of those
  uint32_t min_key;
  uint32_t first;              // first index of the largest logit
  uint32_t listed[2];          // tokens in the lists
  // results, written by one thread
  uint32_t bin, at;
  u64 above_w;
  uint32_t above_n;
};

template <typename T, int NB, int TH>
class Sampler {
 public:
  static constexpr int P = 16 / sizeof(T);  // logits of a 16-byte run
  static constexpr int kWarps = TH / 32;
  __device__ Sampler(const SampleArgs& a, SampleSmem<NB>& sm, T* x)
      : a_(a), sm_(sm), x_(x), cl_(cg::this_cluster()), tid_(threadIdx.x), lane_(threadIdx.x & 31),
        warp_(threadIdx.x >> 5), rank_(NB == 1 ? 0 : cl_.block_rank()), row_(blockIdx.x / NB) {}

  __device__ void run() {
    load();
    // settings, read before the barrier
    const float temp = a_.temperature ? a_.temperature[row_] : 1.0f;
    const int top_k = a_.top_k ? a_.top_k[row_] : 0;
    const float top_p = a_.top_p ? a_.top_p[row_] : 1.0f, min_p = a_.min_p ? a_.min_p[row_] : 0.0f;
    const float u = a_.uniform[row_];
    // log2(e) / T as kh + kl
    const float l2e = 1.44269502f, l2e_lo = 1.92596299e-8f;
    const float kh = l2e / temp, kl = (fmaf(-kh, temp, l2e) + l2e_lo) / temp;
    sync();
    float mx = -INFINITY, mn = INFINITY;
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      const float2 e = *at(&sm_.ext, r);
      mx = fmaxf(mx, e.x);
      mn = fminf(mn, e.y);
    }
    const bool none = !(mx > -INFINITY);
    if (none || !(temp > 0.f) || isinf(kh)) {  // nothing to draw, or the first largest logit
      greedy(mx, none);
      sync();  // no block leaves while another reads its shared memory
      return;
    }
    w_ = Weight{mx, kh, isfinite(kl) ? kl : 0.f, sm_.table};
    // bins over the row's own spread of t; equal logits all lie in the first
    const float range = w_.t(mn);
    limit_ = range < kMaxT ? range : kMaxT;
    scale_ = limit_ > 1e-30f ? kBins / limit_ : 0.f;
    if (isinf(scale_)) scale_ = 0.f;

    const bool use_k = top_k > 0 && top_k < a_.vocab, use_p = top_p < 1.0f, use_m = min_p > 0.0f;
    // the least weight that min-p keeps (above one: only the first token)
    const u64 least = !use_m ? 0 : (min_p > 1.0f ? (1ull << kOneShift) + 1 : __float2ull_ru(min_p * 1099511627776.0f));
    draw(use_k ? top_k : 0, use_p, top_p, use_m, least, u);
    sync();
  }

 private:
  __device__ void sync() {
    if (NB == 1) __syncthreads();
    else cl_.sync();
  }
  template <typename V>
  __device__ V* at(V* p, int r) const {
    return NB == 1 ? p : cl_.map_shared_rank(p, r);
  }

  // The slice into shared memory, tokens that are not allowed as NaN (which maxima, minima and comparisons
  // pass over), and its largest and least logit.
  __device__ void load() {
    const T* g = reinterpret_cast<const T*>(a_.logits) + (int64_t)row_ * a_.ld;
    const int runs = (a_.vocab + P - 1) / P, per = (runs + NB - 1) / NB;
    v0_ = min(a_.vocab, rank_ * per * P);
    n_ = min(a_.vocab, v0_ + per * P) - v0_;
    g += v0_;
    const uint32_t* bits = a_.allowed ? a_.allowed + (int64_t)row_ * ((a_.vocab + 31) / 32) : nullptr;
    const bool wide = (reinterpret_cast<uintptr_t>(g) & 15) == 0;
    const T nan = nan_();
    float mx = -INFINITY, mn = INFINITY;
    constexpr int U = 4;  // runs in flight per thread
    for (int c0 = tid_; c0 * P < n_; c0 += U * TH) {
      alignas(16) T v[U][P];
      uint32_t ok[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i0 = (c0 + k * TH) * P, live = min(P, n_ - i0);
        ok[k] = 0xffffffffu;
        if (live <= 0) continue;
        // a run's bits lie in one word: P divides 32, v0 is a multiple of P
        if (bits) ok[k] = bits[(v0_ + i0) >> 5] >> ((v0_ + i0) & 31);
        if (wide && live == P) {
          *reinterpret_cast<uint4*>(v[k]) = ldg_stream_u4(g + i0);
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) v[k][i] = i < live ? g[i0 + i] : nan;
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int c = c0 + k * TH;
        if (c * P >= n_) continue;
        if (bits) {
#pragma unroll
          for (int i = 0; i < P; ++i)
            if (!((ok[k] >> i) & 1)) v[k][i] = nan;
        }
        extremes(v[k], mx, mn);
        *reinterpret_cast<uint4*>(x_ + c * P) = *reinterpret_cast<const uint4*>(v[k]);
      }
    }
    // the tables, while the loads are on their way
    for (int i = tid_; i < (int)((sizeof(sm_.w1) + sizeof(sm_.c1)) / 16); i += TH)
      reinterpret_cast<uint4*>(&sm_)[i] = make_uint4(0, 0, 0, 0);
    if (tid_ < 256) sm_.table[tid_] = make_uint2(kExpTable.v[tid_], __float_as_uint((float)kExpTable.v[tid_]));
    mx = warp_max(mx);
    mn = warp_min(mn);
    if (lane_ == 0) sm_.red_c[warp_] = __float_as_uint(mx), sm_.red_d[warp_] = __float_as_uint(mn);
    __syncthreads();
    if (warp_ == 0) {
      mx = warp_max(lane_ < kWarps ? __uint_as_float(sm_.red_c[lane_]) : -INFINITY);
      mn = warp_min(lane_ < kWarps ? __uint_as_float(sm_.red_d[lane_]) : INFINITY);
      if (lane_ == 0) {
        sm_.ext = make_float2(mx, mn);
        sm_.first = 0xffffffffu;
        sm_.listed[0] = sm_.listed[1] = 0;
      }
    }
  }
  __device__ static __half nan_h() { return __ushort_as_half(0x7FFF); }
  __device__ static T nan_() {
    if constexpr (sizeof(T) == 2) return nan_h();
    else return __int_as_float(0x7fc00000);
  }
  __device__ static void extremes(const T (&v)[P], float& mx, float& mn) {
    if constexpr (sizeof(T) == 2) {
      const __half2* h = reinterpret_cast<const __half2*>(v);
      const __half2 a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
      const __half2 b = __hmin2(__hmin2(h[0], h[1]), __hmin2(h[2], h[3]));
      const float2 fa = __half22float2(a), fb = __half22float2(b);
      mx = fmaxf(mx, fmaxf(fa.x, fa.y));
      mn = fminf(mn, fminf(fb.x, fb.y));
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) mx = fmaxf(mx, v[i]), mn = fminf(mn, v[i]);
    }
  }

  // f(logit, index in the slice) over the slice, whole 16-byte runs per thread.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int c = tid_; c * P < n_; c += TH) {
      alignas(16) T v[P];
      *reinterpret_cast<uint4*>(v) = reinterpret_cast<const uint4*>(x_)[c];
#pragma unroll
      for (int i = 0; i < P; ++i) f(as_float(v[i]), c * P + i);
    }
  }
  // Bin of t (which is in 0 .. limit); the tokens outside, NaN among them, are those of t > limit_.
  __device__ __forceinline__ int bin_of(float t) const { return min(kBins - 1, (int)(t * scale_)); }
  __device__ __forceinline__ bool inside(float x, float t) const { return t <= limit_ || x == w_.mx; }
  __device__ __forceinline__ int bin_at(float x, float t) const { return x == w_.mx ? 0 : bin_of(t); }

  __device__ void greedy(float mx, bool none) {
    if (!none) {
      uint32_t first = 0xffffffffu;
      each([&](float x, int i) {
        if (x == mx) first = min(first, (uint32_t)(v0_ + i));
      });
      first = __reduce_min_sync(0xffffffffu, first);
      if (lane_ == 0) atomicMin(&sm_.first, first);
      sync();
    }
    if (rank_ == 0 && tid_ == 0) {
      uint32_t first = 0xffffffffu;
#pragma unroll
      for (int r = 0; r < NB; ++r) first = min(first, *at(&sm_.first, r));
      a_.token[row_] = none ? -1 : (int32_t)first;
      if (a_.prob) a_.prob[row_] = none ? __int_as_float(0x7fc00000) : 1.0f;
    }
  }

  // Inclusive sums over the block of one (count, weight) a thread.
  __device__ void scan(uint32_t& c, u64& w) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t cu = __shfl_up_sync(0xffffffffu, c, o);
      const u64 wu = __shfl_up_sync(0xffffffffu, w, o);
      if (lane_ >= o) c += cu, w += wu;
    }
    if (lane_ == 31) sm_.red_c[warp_] = c, sm_.red_w[warp_] = w;
    __syncthreads();
    uint32_t cb = lane_ < warp_ ? sm_.red_c[lane_] : 0;
    u64 wb = lane_ < warp_ ? sm_.red_w[lane_] : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      cb += __shfl_xor_sync(0xffffffffu, cb, o);
      wb += __shfl_xor_sync(0xffffffffu, wb, o);
    }
    c += cb, w += wb;
    __syncthreads();
  }

  template <int N>
  __device__ u64 limbs_at(Limbs<N>& h, int b, int r) const {
    return (u64)*at(&h.v[0][b], r) + ((u64)*at(&h.v[1][b], r) << 14) + ((u64)*at(&h.v[2][b], r) << 28);
  }

  // The blocks' histograms added up, and the running sums above every bin: na, and wa with weights.
  __device__ void combine(bool weights) {
    constexpr int share = kBins / NB, per = kBins / TH;
    sync();
    if (NB > 1) {
      for (int i = tid_; i < share; i += TH) {
        const int b = rank_ * share + i;
        uint32_t c = 0;
        u64 w = 0;
#pragma unroll
        for (int r = 0; r < NB; ++r) {
          c += *at(&sm_.c1[b], r);
          if (weights) w += limbs_at(sm_.w1, b, r);
        }
        sm_.own_n[i] = c;
        sm_.own_w[i] = w;
      }
      sync();
    }
    uint32_t c[per], cs = 0;
    u64 w[per], ws = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const int b = tid_ * per + i;
      if (NB == 1) {
        c[i] = sm_.c1[b];
        w[i] = weights ? limbs_at(sm_.w1, b, 0) : 0;
      } else {
        c[i] = *at(&sm_.own_n[b % share], b / share);
        w[i] = weights ? *at(&sm_.own_w[b % share], b / share) : 0;
      }
      cs += c[i], ws += w[i];
    }
    uint32_t ci = cs;
    u64 wi = ws;
    scan(ci, wi);
    ci -= cs, wi -= ws;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const int b = tid_ * per + i;
      sm_.na[b] = ci, sm_.wa[b] = wi;
      ci += c[i], wi += w[i];
    }
    if (tid_ == TH - 1) sm_.na[kBins] = ci, sm_.wa[kBins] = wi;
    __syncthreads();
  }

  // The bin in which the running count (or weight) reaches target, which the row's does.
  __device__ int find_bin(bool by_count, u64 target) {
    for (int b = tid_; b < kBins; b += TH) {
      const u64 lo = by_count ? sm_.na[b] : sm_.wa[b], hi = by_count ? sm_.na[b + 1] : sm_.wa[b + 1];
      if (lo < target && target <= hi) sm_.bin = b;
    }
    __syncthreads();
    const int b = sm_.bin;
    __syncthreads();
    return b;
  }

  // The row's tokens of bins b0 .. b1 (n of them, at most kCap) into cand, sorted, with their running weights
  // from `above` on in cum. list: 0 or 1, each used once.
  __device__ void gather(int b0, int b1, int n, int list, u64 above) {
    u64* mine = reinterpret_cast<u64*>(&sm_.w1) + list * kCap;
    static_assert(sizeof(sm_.w1) >= 2 * kCap * sizeof(u64), "the lists lie over the histogram");
    each([&](float x, int i) {
      const float t = w_.t(x);
      if (!inside(x, t)) return;
      const int b = bin_at(x, t);
      if (b < b0 || b > b1) return;
      const uint32_t key = key_of(x);
      if (key < floor_) return;
      const uint32_t k = atomicAdd(&sm_.listed[list], 1u);
      if (k < (uint32_t)kCap) mine[k] = ((u64)key << 32) | (uint32_t)~(v0_ + i);
    });
    sync();
    int off = 0;
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      const int c = (int)*at(&sm_.listed[list], r);
      for (int i = tid_; i < c; i += TH)
        if (off + i < kCap) sm_.cand[off + i] = *at(mine + i, r);
      off += c;
    }
    int m = 32;
    while (m < n) m *= 2;
    for (int i = n + tid_; i < m; i += TH) sm_.cand[i] = 0;
    __syncthreads();
    // falling order, bitonic; up to a distance of 32 a warp's pairs stay within its own 64 places
    for (int k = 2; k <= m; k *= 2)
      for (int j = k / 2; j; j /= 2) {
        for (int p = tid_; p < m / 2; p += TH) {
          const int i = 2 * p - (p & (j - 1)), l = i + j;
          const u64 x = sm_.cand[i], y = sm_.cand[l];
          if ((x < y) == ((i & k) == 0)) sm_.cand[i] = y, sm_.cand[l] = x;
        }
        if (j > 32 || (j == 1 && k >= 64)) __syncthreads();
        else __syncwarp();
      }
    __syncthreads();
    // running weights
    constexpr int per = kCap / TH;
    u64 w[per], ws = 0;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const int q = tid_ * per + i;
      w[i] = q < n ? w_(value_of((uint32_t)(sm_.cand[q] >> 32))) : 0;
      ws += w[i];
    }
    u64 wi = ws;
    scan(c, wi);
    wi += above - ws;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      wi += w[i];
      sm_.cum[tid_ * per + i] = wi;
    }
    __syncthreads();
  }

  // First of n gathered tokens whose running weight reaches target (the last if none does).
  __device__ int reach(int n, u64 target, u64 above) {
    if (tid_ == 0) sm_.at = n - 1;
    __syncthreads();
    for (int i = tid_; i < n; i += TH)
      if (sm_.cum[i] >= target && (i ? sm_.cum[i - 1] : above) < target) sm_.at = i;
    __syncthreads();
    const int i = sm_.at;
    __syncthreads();
    return i;
  }

  // The place where the running count or weight of bin b reaches target, by a radix descent over the bin's keys:
  // any number of tokens, any ties.
  __device__ Place descend(bool by_count, int b, u64 target) {
    if (tid_ == 0) sm_.above_n = sm_.na[b], sm_.above_w = sm_.wa[b];
    sync();  // what the histograms lie over is no longer read
    for (int i = tid_; i < (int)(sizeof(sm_.wd) / 4); i += TH) reinterpret_cast<uint32_t*>(&sm_.wd)[i] = 0;
    for (int i = tid_; i < (int)(sizeof(sm_.cd) / 4); i += TH) reinterpret_cast<uint32_t*>(&sm_.cd)[i] = 0;
    __syncthreads();
    uint32_t prefix = 0;
#pragma unroll 1
    for (int d = 0; d < kDigits; ++d) {
      const int shift = 24 - 8 * d;
      each([&](float x, int) {
        const float t = w_.t(x);
        if (!inside(x, t) || bin_at(x, t) != b) return;
        const uint32_t k = key_of(x);
        if (k < floor_ || (d && (k >> (shift + 8)) != prefix)) return;
        const int g = (k >> shift) & 255;
        atomicAdd(&sm_.cd[d][g], 1u);
        if (d < kDigits - 1) sm_.wd[d].add(g, w_(x));
      });
      sync();
      // digits from the top, one a thread; all threads take part in the scan
      const int g = 255 - tid_;
      uint32_t c = 0;
      u64 w = 0;
      if (g >= 0) {
#pragma unroll
        for (int r = 0; r < NB; ++r) {
          c += *at(&sm_.cd[d][g], r);
          w += limbs_at(sm_.wd[d], g, r);
        }
        if (d == kDigits - 1 && c) w = c * w_(value_of((prefix << 8) | g));
      }
      uint32_t ci = c;
      u64 wi = w;
      const uint32_t an = sm_.above_n;
      const u64 aw = sm_.above_w;
      scan(ci, wi);
      const u64 lo = by_count ? an + ci - c : aw + wi - w, hi = by_count ? an + ci : aw + wi;
      if (g >= 0 && lo < target && target <= hi) sm_.bin = g, sm_.above_n = an + ci - c, sm_.above_w = aw + wi - w;
      __syncthreads();
      prefix = (prefix << 8) | sm_.bin;
      __syncthreads();
    }
    Place p;
    p.key = prefix;
    p.above_w = sm_.above_w;
    p.index = -1;
    const u64 one = w_(value_of(prefix));
    p.tie = by_count ? (uint32_t)(target - sm_.above_n) : (uint32_t)((target - p.above_w + one - 1) / one);
    sync();  // the digit histograms are read before a next descent clears them
    return p;
  }

  // Writes token and probability of tie number p.tie of key p.key, whichever block holds it.
  __device__ void locate(const Place& p, u64 total) {
    // every block's count of the key, over its threads' contiguous parts
    const int per = (n_ + TH - 1) / TH, i0 = min(n_, tid_ * per), i1 = min(n_, i0 + per);
    const float v = value_of(p.key);
    uint32_t mine = 0;
    for (int i = i0; i < i1; ++i) mine += as_float(x_[i]) == v;
    uint32_t incl = mine;
    u64 none = 0;
    scan(incl, none);
    if (tid_ == TH - 1) sm_.listed[0] = incl;
    sync();
    uint32_t before = incl - mine;
    for (int r = 0; r < rank_; ++r) before += *at(&sm_.listed[0], r);
    if (before < p.tie && p.tie <= before + mine)
      for (int i = i0; i < i1; ++i)
        if (as_float(x_[i]) == v && ++before == p.tie) {
          write(v0_ + i, p.key, total);
          break;
        }
  }
  __device__ void write(int32_t index, uint32_t key, u64 total) {
    a_.token[row_] = index;
    if (a_.prob) a_.prob[row_] = (float)((double)w_(value_of(key)) / (double)total);
  }

  __device__ static u64 part_of(float share, u64 total) {  // smallest sum that is at least `share` of total
    const double t = ceil((double)share * (double)total);
    return t >= 1.0 ? min((u64)t, total) : 1ull;
  }
  __device__ static u64 beyond(float u, u64 total) {  // smallest sum above u times total
    const double t = floor((double)u * (double)total);
    return t >= 0.0 ? min((u64)t + 1, total) : 1ull;
  }

  __device__ void draw(int k, bool use_p, float top_p, bool use_m, u64 least, float u) {
    u64 total = 0;  // weight of what the cuts so far keep
    bool cut_k = false;
    if (k) {
      each([&](float x, int) {
        const float t = w_.t(x);
        if (inside(x, t)) atomicAdd(&sm_.c1[bin_at(x, t)], 1u);
      });
      combine(false);
      if (sm_.na[kBins] > (uint32_t)k) {
        const int b = find_bin(true, k), n = sm_.na[b + 1];
        if (n <= kCap) {  // the first k tokens and the rest of their last bin: everything else happens on them
          gather(0, b, n, 0, 0);
          int keep = k;
          if (use_p) keep = min(keep, reach(keep, part_of(top_p, sm_.cum[keep - 1]), 0) + 1);
          if (use_m) {
            // tokens of at least min-p's weight: those before the first lighter one
            if (tid_ == 0) sm_.at = 0xffffffffu;
            __syncthreads();
            for (int i = tid_; i < keep; i += TH)
              if (sm_.cum[i] - (i ? sm_.cum[i - 1] : 0) < least) atomicMin(&sm_.at, (uint32_t)i);
            __syncthreads();
            const uint32_t m = sm_.at;
            __syncthreads();
            keep = min((uint32_t)keep, max(m, 1u));
          }
          total = sm_.cum[keep - 1];
          const int i = reach(keep, beyond(u, total), 0);
          if (rank_ == 0 && tid_ == 0) write((int32_t)~(uint32_t)sm_.cand[i], (uint32_t)(sm_.cand[i] >> 32), total);
          return;
        }
        const Place p = descend(true, b, k);
        floor_ = p.key;
        cut_k = true;
      }
      // the histogram again, with weights
      sync();
      for (int i = tid_; i < kBins; i += TH) sm_.c1[i] = 0;
      __syncthreads();
    }
    u64 m_sum = 0;
    uint32_t m_key = 0xffffffffu;
    each([&](float x, int) {
      const float t = w_.t(x);
      if (!inside(x, t)) return;
      const uint32_t key = key_of(x);
      if (key < floor_) return;
      const u64 w = w_(x);
      const int b = bin_at(x, t);
      sm_.w1.add(b, w);
      atomicAdd(&sm_.c1[b], 1u);
      if (use_m && w >= least) m_sum += w, m_key = min(m_key, key);
    });
    if (use_m) {
      uint32_t c = 0;
      scan(c, m_sum);
      m_key = __reduce_min_sync(0xffffffffu, m_key);
      if (lane_ == 0) sm_.red_d[warp_] = m_key;
      __syncthreads();
      if (tid_ == TH - 1) {
        for (int i = 0; i < kWarps; ++i) m_key = min(m_key, sm_.red_d[i]);
        sm_.min_sum = m_sum;
        sm_.min_key = m_key;
      }
    }
    combine(true);
    if (use_m) {
      m_sum = 0, m_key = 0xffffffffu;
#pragma unroll
      for (int r = 0; r < NB; ++r) {
        m_sum += *at(&sm_.min_sum, r);
        m_key = min(m_key, *at(&sm_.min_key, r));
      }
    }
    // what top-k keeps: all at or above its last key, without the ties past its last token
    uint32_t end_key = floor_;
    total = sm_.wa[kBins];
    if (cut_k) total -= w_(value_of(floor_)) * (sm_.na[kBins] - (uint32_t)k);
    int held = -1;  // the bin whose tokens are gathered
    if (use_p) {
      const u64 target = part_of(top_p, total);
      const int b = find_bin(false, target), n = sm_.na[b + 1] - sm_.na[b];
      if (n <= kCap) {
        gather(b, b, n, 0, sm_.wa[b]);
        const int i = reach(n, target, sm_.wa[b]);
        total = sm_.cum[i];
        end_key = (uint32_t)(sm_.cand[i] >> 32);
        held = b;
      } else {
        const Place p = descend(false, b, target);
        total = p.above_w + p.tie * w_(value_of(p.key));
        end_key = p.key;
      }
    }
    if (use_m) {
      if (m_key == 0xffffffffu) total = 1ull << kOneShift;  // min-p above one
      else if (m_key > end_key) total = m_sum;
    }
    const u64 target = beyond(u, total);
    const int b = find_bin(false, target), n = sm_.na[b + 1] - sm_.na[b];
    if (n <= kCap) {
      if (b != held) gather(b, b, n, 1, sm_.wa[b]);
      const int i = reach(n, target, sm_.wa[b]);
      if (rank_ == 0 && tid_ == 0) write((int32_t)~(uint32_t)sm_.cand[i], (uint32_t)(sm_.cand[i] >> 32), total);
    } else {
      locate(descend(false, b, target), total);
    }
  }

  const SampleArgs& a_;
  SampleSmem<NB>& sm_;
  T* x_;
  cg::cluster_group cl_;
  const int tid_, lane_, warp_, rank_, row_;
  int v0_ = 0, n_ = 0;
  Weight w_{};
  float limit_ = 0.f, scale_ = 0.f;
  uint32_t floor_ = 0;  // keys below are cut off (top-k by descent)
};

template <typename T, int NB, int TH>
__global__ void __launch_bounds__(TH, 1) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SampleSmem<NB>& sm = *reinterpret_cast<SampleSmem<NB>*>(smem_raw);
  T* x = reinterpret_cast<T*>(smem_raw + (sizeof(SampleSmem<NB>) + 15) / 16 * 16);
  Sampler<T, NB, TH>(a, sm, x).run();
}

template <typename T, int NB, int TH>
cudaError_t launch_sample_th(cudaStream_t s, const SampleArgs& a, size_t slice) {
  const size_t smem = (sizeof(SampleSmem<NB>) + 15) / 16 * 16 + slice;
  cudaError_t e =
      cudaFuncSetAttribute(sample_kernel<T, NB, TH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * NB));
  cfg.blockDim = dim3(TH);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = NB;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, NB, TH>, a);
}
template <typename T, int NB>
cudaError_t launch_sample_nb(cudaStream_t s, const SampleArgs& a, size_t slice) {
  // a slice of more than 16 tokens a thread: twice the threads
  return slice / sizeof(T) > 512 * 32 ? launch_sample_th<T, NB, 1024>(s, a, slice)
                                      : launch_sample_th<T, NB, 512>(s, a, slice);
}

template <typename T>
cudaError_t launch_sample_t(cudaStream_t s, const SampleArgs& a) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  auto slice = [&](int nb) {
    constexpr int P = 16 / sizeof(T);
    const int runs = (a.vocab + P - 1) / P;
    return (size_t)((runs + nb - 1) / nb) * 16;
  };
  // as many blocks to a row as there are SMs for, each with at least 4 KB of it
  int nb = 1;
  while (nb < kMaxCluster && (slice(nb) > kKeyBytes || ((int64_t)a.rows * nb * 2 <= n_sm && slice(nb) > 4096))) nb *= 2;
  if (slice(nb) > kKeyBytes) return cudaErrorInvalidValue;
  switch (nb) {
    case 1: return launch_sample_nb<T, 1>(s, a, slice(nb));
    case 2: return launch_sample_nb<T, 2>(s, a, slice(nb));
    case 4: return launch_sample_nb<T, 4>(s, a, slice(nb));
    default: return launch_sample_nb<T, 8>(s, a, slice(nb));
  }
}

}  // namespace

int64_t sample_max_vocab(bool f32) { return (int64_t)kMaxCluster * (kKeyBytes / (f32 ? 4 : 2)); }

cudaError_t launch_sample(cudaStream_t s, const SampleArgs& a) {
  if (a.rows < 1 || a.vocab < 1 || a.vocab > sample_max_vocab(a.f32)) return cudaErrorInvalidValue;
  return a.f32 ? launch_sample_t<float>(s, a) : launch_sample_t<__half>(s, a);
}

}  // namespace mag
