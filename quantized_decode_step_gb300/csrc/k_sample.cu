// Sampling of the next token from rows of logits: temperature, top-k, top-p and min-p, with given random numbers.
//
// The tokens of a row stand in order (logit falling, equal logits by index rising); w_i = exp((l_i - max) / T) and
// every cut keeps a prefix of that order: top-k its first k tokens, top-p the shortest prefix of those whose w add
// up to top_p of theirs, min-p the tokens with w >= min_p. The token is the first of the shortest prefix whose
// running sum of w passes u times the prefix's sum.
//
// A row is never sorted. Its tokens fall into 2,048 bins by t = (max - l) log2(e) / T, so the bins stand in the
// tokens' order. With top-k the bins that hold the first k tokens are gathered and sorted, and everything else
// happens on those: the bins above the k-th largest of a few thousand partial maxima, if that is few enough
// tokens, or what counting all bins says. Without, every bin's weights are added up; the end of top-p and the token each
// lie in one bin, found on the bins' running sums, whose tokens are gathered and sorted. A bin of more than kCap
// tokens, mostly equal logits, is searched by a radix descent over the logits as ordered integers instead.
//
// The weights are integers, w in units of 2^-40 to within 2^-30 of their value (a table of 2^(-j/256), a cubic for the
// rest, t in two fp32 terms), so that their sums are exact in 64 bits: no order of atomics changes a result,
// sums over different sets of the same tokens agree to the last unit, and a token differs from that of real
// arithmetic only where u falls within about 1e-9 / sqrt(tokens) of a border.
//
// What bounds it: the logits are read once from HBM (256 rows of 128,256 in fp16: 10 us), so with few rows the
// latency of the passes between cluster barriers, with many the passes' waits for the row from L2 and the
// instructions and shared-memory adds of a token: about 7 and 1 to count it, 30 and 2 or 3 for its weight. With few
// rows a cluster of blocks shares a row, each with its slice in shared memory, as many blocks as the row count
// leaves SMs for; with many a block has a row and later passes read it from L2: two blocks an SM, or one where long
// fp16 rows are counted by value (132 KB of counts).
#include <cooperative_groups.h>

#include <algorithm>

#include "kernels.h"

namespace mag {

namespace {

namespace cg = cooperative_groups;

typedef unsigned long long u64;

constexpr int kBins = 2048, kDead = kBins - 1;  // the last bin: tokens that cannot be drawn, or weigh nothing
constexpr float kMagic = 12582912.0f;    // 1.5 2^23: adding it leaves a number's integer part in the low bits
constexpr int kMagicBits = 0x4B400000;
constexpr int kCap = 2048;             // most tokens gathered and sorted
constexpr int kMaxCluster = 8;
constexpr size_t kKeyBytes = 132 * 1024;  // most bytes of a slice in shared memory
constexpr int kOneShift = 40;          // w = 1 is 2^40
constexpr float kMaxT = 41.0f;         // tokens of t >= 41 weigh less than half a unit
constexpr int kDigits = 4, kDigitBins = 256;

// 2^(-j / 256) in units of 2^-31, j = 0 .. 255.
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

// w / total to one rounding: both as two fp32 terms, the quotient corrected by its remainder.
__device__ float quotient(u64 w, u64 total) {
  const float wh = __ull2float_rn(w), wl = __ll2float_rn((long long)(w - __float2ull_rn(wh)));
  const float th = __ull2float_rn(total), tl = __ll2float_rn((long long)(total - __float2ull_rn(th)));
  const float q = wh / th;
  return q + (fmaf(-q, th, wh) + fmaf(-q, tl, wl)) / th;
}

// exp((x - max) / T) in units of 2^-40, of t = (max - x) (kh + kl) below kMaxT; kh + kl = log2(e) / T. Without a branch, so
// that several tokens' run side by side.
constexpr float kDeadT = 41.99f;   // t of a token that cannot be drawn; it weighs 0
struct Weight {
  float mx, kh, kl;
  const uint2* table;
  __device__ __forceinline__ float t(float x) const { return fminf(__fmul_rn(__fsub_rn(mx, x), kh), kDeadT); }
  // w = m 2^(9 - sh), sh = t's whole part. bits: its low 8 bits and the 5 above are the table's index and sh - 10.
  // kExact: max - x with its rounding error, which logits in fp32 have wherever the maximum is larger; in fp16 the difference
  // is exact but for logits below 2^-11 of it, and then off by 2^-24 of itself.
  template <bool kExact>
  __device__ __forceinline__ void split(float x, float th, uint32_t& m, int& bits) const {
    const float s = __fsub_rn(mx, x);
    float tl = fmaf(s, kl, fmaf(s, kh, -th));  // t = th + tl
    if (kExact) {
      const float bb = __fsub_rn(s, mx);
      tl = fmaf(__fsub_rn(__fsub_rn(mx, __fsub_rn(s, bb)), __fadd_rn(x, bb)), kh, tl);
    }
    // th = i / 256 + ..: i, and below the integer part of a product, by adding a number of ulp 1
    constexpr float kBase = kMagic - 2560.0f;
    const float im = fmaf(th, 256.0f, kBase);
    const float r = fmaf(im - kBase, 0.00390625f, -th) - tl;  // 2^-(th + tl) = 2^(-i / 256) 2^r
    const float c = r * fmaf(r, fmaf(r, 5.5504109e-2f, 0.24022651f), 0.69314718f);
    bits = __float_as_int(im);  // kMagicBits + i - 2560
    const uint2 w0 = table[bits & 255];
    m = w0.x + (__float_as_int(fmaf(__uint_as_float(w0.y), c, kMagic)) - kMagicBits);
  }
  // sh >= 10 (and below 42), the value at most 2^30
  __device__ __forceinline__ static uint32_t small(uint32_t m, int bits) {
    return (__funnelshift_r(m, 0u, (uint32_t)(bits >> 8)) + 1u) >> 1;
  }
  __device__ __forceinline__ static u64 any(uint32_t m, int bits) {
    const int sh = ((bits - kMagicBits) >> 8) + 10;
    return sh < 10 ? (u64)m << (9 - max(sh, 0)) : (u64)small(m, bits);
  }
  template <bool kExact>
  __device__ __forceinline__ u64 value(float x) const {
    uint32_t m;
    int bits;
    split<kExact>(x, t(x), m, bits);
    return any(m, bits);
  }
  // The weight over total, before the weight's rounding to units: that would leave a token of 2^-28 of the largest one's
  // weight a probability of 12 bits.
  template <bool kExact>
  __device__ float share(float x, u64 total) const {
    uint32_t m;
    int bits;
    split<kExact>(x, t(x), m, bits);
    return ldexpf(quotient(m, total), 9 - (((bits - kMagicBits) >> 8) + 10));
  }
};

// A histogram of weights: 64-bit adds to shared memory are compare-and-swap loops (59 clocks a warp on logits' bins, 1,700
// on one bin), 32-bit adds take 2.4 to 3.3 clocks whatever the bins. So a weight goes in as limbs of 15, 15 and 11
// bits, the third of the few tokens of t < 10; a slice has fewer than 2^17 tokens, so a limb's sum (a limb is at most
// 2^15) stays below 2^32.
constexpr int kMaxSlice = (1 << 17) - 1;
template <int N>
struct Limbs {
  uint32_t v[3][N];
  __device__ __forceinline__ void add(int b, u64 w) {
    atomicAdd(&v[0][b], (uint32_t)w & 0x7FFFu);
    atomicAdd(&v[1][b], (uint32_t)(w >> 15) & 0x7FFFu);
    atomicAdd(&v[2][b], (uint32_t)(w >> 30));
  }
  __device__ __forceinline__ void add_small(int b, uint32_t w) {  // at most 2^30
    atomicAdd(&v[0][b], w & 0x7FFFu);
    atomicAdd(&v[1][b], w >> 15);
  }
};

// share * total as (whole part, whether there is more), share in (0, 1)
__device__ u64 times(float share, u64 total, bool& more) {
  const uint32_t b = __float_as_uint(share);
  const int e = max(1, (int)(b >> 23));
  const u64 m = (b & 0x7FFFFFu) | (b >> 23 ? 0x800000u : 0u);  // share = m 2^(e - 150)
  const u64 hi = __umul64hi(m, total), lo = m * total;
  const int sh = 150 - e;  // 24 ..
  u64 whole = 0, rest;
  if (sh < 64) {
    whole = (hi << (64 - sh)) | (lo >> sh);
    rest = lo << (64 - sh);
  } else {
    whole = sh < 128 ? hi >> (sh - 64) : 0;
    rest = lo | (sh < 128 ? (sh > 64 ? hi << (128 - sh) : 0) : hi);
  }
  more = rest != 0;
  return whole;
}
__device__ u64 part_of(float share, u64 total) {  // smallest sum that is at least `share` of total
  if (!(share > 0.f)) return 1;
  bool more;
  const u64 t = times(share, total, more);
  return max((u64)1, min(total, t + more));
}
__device__ u64 beyond(float u, u64 total) {  // smallest sum above u times total
  if (!(u > 0.f)) return 1;
  if (u >= 1.f) return total;
  bool more;
  return min(total, times(u, total, more) + 1);
}

// The settings of a row.
struct Settings {
  float temp, top_p, min_p, u;
  int top_k;
  float kh, kl;    // log2(e) / T
  bool greedy;     // the first of the largest logits
  bool use_p, use_m;
  u64 least;       // the least weight that min-p keeps (above one: only the first token)
  __device__ Settings(const SampleArgs& a, int row)
      : temp(a.temperature ? a.temperature[row] : 1.0f), top_p(a.top_p ? a.top_p[row] : 1.0f),
        min_p(a.min_p ? a.min_p[row] : 0.0f), u(a.uniform[row]), top_k(a.top_k ? a.top_k[row] : 0) {
    const float l2e = 1.44269502f, l2e_lo = 1.92596299e-8f;
    kh = l2e / temp;
    kl = (fmaf(-kh, temp, l2e) + l2e_lo) / temp;
    if (!isfinite(kl)) kl = 0.f;
    greedy = !(temp > 0.f) || isinf(kh);
    if (top_k <= 0 || top_k >= a.vocab) top_k = 0;
    use_p = top_p < 1.0f;
    use_m = min_p > 0.0f;
    least = !use_m ? 0 : (min_p > 1.0f ? (1ull << kOneShift) + 1 : __float2ull_ru(min_p * 1099511627776.0f));
  }
};

struct Place {      // a place in the falling order: token `index`, or tie number `tie` (from 1) of key `key`
  u64 above_w;      // weight before its tie 1 (by index: up to and with the token, tie 0)
  uint32_t key, tie;
  int32_t index;    // the token, -1 where only key and tie are known
};

template <int NB>
struct SampleSmem {
  Limbs<kBins> w1;   // this block's histograms (of weights, of counts); later two lists of gathered tokens
  uint32_t c1[kBins];
  union {            // zero up to here at the start
    struct {         // weights: the row's bins that this block adds up
      u64 own_w[NB == 1 ? 1 : kBins / NB];
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
  uint2 table[256];            // 2^(-j / 256) in units of 2^-31, and as a float
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
  uint32_t tokens;             // this block's tokens that weigh anything
};

// ST: the slice is kept in shared memory; otherwise (NB = 1) later passes read it again.
template <typename T, int NB, int TH, bool ST>
class Sampler {
 public:
  static constexpr int P = 16 / sizeof(T);  // logits of a 16-byte run
  static constexpr int kWarps = TH / 32;
  static constexpr bool kExact = sizeof(T) == 4;
  __device__ Sampler(const SampleArgs& a, SampleSmem<NB>& sm, T* x)
      : a_(a), sm_(sm), x_(x), cl_(cg::this_cluster()), tid_(threadIdx.x), lane_(threadIdx.x & 31),
        warp_(threadIdx.x >> 5), rank_(NB == 1 ? 0 : cl_.block_rank()), row_(blockIdx.x / NB) {}

  __device__ void run() {
    load();
    const Settings g(a_, row_);  // before the barrier
    sync();
    float mx = -INFINITY, mn = INFINITY;
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      const float2 e = *at(&sm_.ext, r);
      mx = fmaxf(mx, e.x);
      mn = fminf(mn, e.y);
    }
    const bool none = !(mx > -INFINITY);
    if (none || g.greedy) {  // nothing to draw, or the first largest logit
      greedy(mx, none);
      sync();  // no block leaves while another reads its shared memory
      return;
    }
    if (mx == INFINITY) {  // infinite logits share all the weight: they become 0, the others none
      infinite_ = true;
      mx = mn = 0.f;
    }
    w_ = Weight{mx, g.kh, g.kl, sm_.table};
    // bins over the row's own spread of t, up to kMaxT; equal logits all lie in the first
    const float limit = fminf(w_.t(mn), kMaxT);
    per_t_ = limit > 0.f ? fminf((kDead - 1) / limit, 3e38f) : 1000.f;

    draw(g.top_k, g.use_p, g.top_p, g.use_m, g.least, g.u);
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

  // f(run of P logits as they lie, its number c) over the slice, U runs in flight per thread; tokens that are not
  // allowed are NaN (which maxima, minima and comparisons pass over).
  template <int U, typename F>
  __device__ __forceinline__ void from_global(F f) const {
    const T* g = reinterpret_cast<const T*>(a_.logits) + (int64_t)row_ * a_.ld + v0_;
    const uint32_t* bits = a_.allowed ? a_.allowed + (int64_t)row_ * ((a_.vocab + 31) / 32) : nullptr;
    const bool wide = (reinterpret_cast<uintptr_t>(g) & 15) == 0;
    const T nan = nan_();
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
          *reinterpret_cast<uint4*>(v[k]) = ST ? ldg_stream_u4(g + i0) : __ldg(reinterpret_cast<const uint4*>(g + i0));
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) v[k][i] = i < live ? g[i0 + i] : nan;
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int c = c0 + k * TH;
        if (c * P >= n_) continue;
        if (bits) {  // all of a number's bits but the sign set: NaN
          uint32_t* w = reinterpret_cast<uint32_t*>(v[k]);
          const uint32_t off = ~ok[k];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (P == 8) w[i] |= (((off >> (2 * i)) & 1u) | (((off >> (2 * i)) & 2u) << 15)) * 0x7FFFu;
            else w[i] |= (uint32_t)((int32_t)(off << (31 - i)) >> 31) & 0x7FFFFFFFu;
          }
        }
        f(v[k], c, k);
      }
    }
  }
  // The row's extremes, and (ST) the slice into shared memory.
  __device__ void load() {
    const int runs = (a_.vocab + P - 1) / P, per = (runs + NB - 1) / NB;
    v0_ = min(a_.vocab, rank_ * per * P);
    n_ = min(a_.vocab, v0_ + per * P) - v0_;
    float mn = INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) part_max_[k] = -INFINITY;
    from_global<4>([&](const T (&v)[P], int c, int k) {
      extremes(v, part_max_[k], mn);
      if (ST) *reinterpret_cast<uint4*>(x_ + c * P) = *reinterpret_cast<const uint4*>(v);
    });
    for (int i = tid_; i < (int)((sizeof(sm_.w1) + sizeof(sm_.c1)) / 16); i += TH)
      reinterpret_cast<uint4*>(&sm_)[i] = make_uint4(0, 0, 0, 0);
    if (tid_ < 256) sm_.table[tid_] = make_uint2(kExpTable.v[tid_], __float_as_uint((float)kExpTable.v[tid_]));
    float mx = warp_max(fmaxf(fmaxf(part_max_[0], part_max_[1]), fmaxf(part_max_[2], part_max_[3])));
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

  // f(run of P logits as they lie, number) over the slice.
  template <typename F>
  __device__ __forceinline__ void raw_runs(F f) const {
    if constexpr (ST) {
      for (int c = tid_; c * P < n_; c += TH) {
        alignas(16) T v[P];
        *reinterpret_cast<uint4*>(v) = reinterpret_cast<const uint4*>(x_)[c];
        f(v, c);
      }
    } else {
      from_global<2>([&](const T (&v)[P], int c, int) { f(v, c); });
    }
  }
  __device__ __forceinline__ void widen(const T (&v)[P], float (&x)[P]) const {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = as_float(v[i]);
    if (infinite_) {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = x[i] == INFINITY ? 0.f : NAN;
    }
  }
  // f(P logits, the first's index in the slice) over the slice.
  template <typename F>
  __device__ __forceinline__ void runs(F f) const {
    raw_runs([&](const T (&v)[P], int c) {
      float x[P];
      widen(v, x);
      f(x, c * P);
    });
  }
  // f(logit, index in the slice).
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    runs([&](const float (&x)[P], int i0) {
#pragma unroll
      for (int i = 0; i < P; ++i) f(x[i], i0 + i);
    });
  }
  // A token's bin is b = coord - kMagic (an integer), which rises with t.
  __device__ __forceinline__ float coord(float t) const { return fminf(fmaf(t, per_t_, kMagic), kMagic + kDead); }
  __device__ __forceinline__ static int bin_at(float coord) { return __float_as_int(coord) - kMagicBits; }
  __device__ __forceinline__ float coord_of(float x) const { return coord(w_.t(x)); }

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

  __device__ __forceinline__ u64 weight(float x) const { return w_.template value<kExact>(x); }

  template <int N>
  __device__ u64 limbs_at(Limbs<N>& h, int b, int r) const {
    return (u64)*at(&h.v[0][b], r) + ((u64)*at(&h.v[1][b], r) << 15) + ((u64)*at(&h.v[2][b], r) << 30);
  }

  // The blocks' counts added up, and the running count above every bin: na.
  __device__ void add_counts() {
    constexpr int per = kBins / TH;
    sync();
    uint32_t c[per] = {}, cs = 0;
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      const uint32_t* p = at(&sm_.c1[tid_ * per], r);
      uint32_t v[per];
      if constexpr (per == 4) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
      else *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
#pragma unroll
      for (int i = 0; i < per; ++i) c[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < per; ++i) cs += c[i];
    uint32_t ci = cs;
    u64 none = 0;
    scan(ci, none);
    ci -= cs;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      sm_.na[tid_ * per + i] = ci;
      ci += c[i];
    }
    if (tid_ == TH - 1) sm_.na[kBins] = ci;
    __syncthreads();
  }
  // The same of the weights: wa. Block r adds up its share of the bins, then everyone takes all of them.
  __device__ void add_weights() {
    constexpr int share = kBins / NB, per = kBins / TH;
    sync();
    if (NB > 1) {
      for (int i = tid_; i < share; i += TH) {
        u64 w = 0;
#pragma unroll
        for (int r = 0; r < NB; ++r) w += limbs_at(sm_.w1, rank_ * share + i, r);
        sm_.own_w[i] = w;
      }
      sync();
    }
    uint32_t none = 0;
    u64 w[per], ws = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const int b = tid_ * per + i;
      if (NB == 1) w[i] = limbs_at(sm_.w1, b, 0);
      else w[i] = *at(&sm_.own_w[b % share], b / share);
      ws += w[i];
    }
    u64 wi = ws;
    scan(none, wi);
    wi -= ws;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      sm_.wa[tid_ * per + i] = wi;
      wi += w[i];
    }
    if (tid_ == TH - 1) sm_.wa[kBins] = wi;
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

  __device__ __forceinline__ void list(int which, float x, int i) {
    u64* mine = reinterpret_cast<u64*>(&sm_.w1) + which * kCap;
    static_assert(sizeof(sm_.w1) + sizeof(sm_.c1) >= 2 * kCap * sizeof(u64), "the lists lie over the histograms");
    const uint32_t key = key_of(x);
    if (key < floor_) return;
    const uint32_t k = atomicAdd(&sm_.listed[which], 1u);
    if (k < (uint32_t)kCap) mine[k] = ((u64)key << 32) | (uint32_t)~(v0_ + i);
  }
  // The row's tokens of bins b0 .. b1 (not the dead one) into a list (each is used once). Most runs have none: a test
  // against bounds of the logits, a little wide, comes first.
  __device__ void gather(int b0, int b1, int which) {
    const float c0 = kMagic + b0, c1 = kMagic + b1;
    const float inv = 1.0f / (per_t_ * w_.kh), wide = fabsf(w_.mx) * 1e-6f;  // logits per bin
    const float hi = b0 ? w_.mx - (b0 - 0.75f) * inv * 0.99999f + wide : INFINITY;
    const float lo = w_.mx - (b1 + 0.75f) * inv * 1.00001f - wide;
    const bool all = infinite_ || !(lo > -INFINITY) || !(inv > 1e-30f);
    const __half2 lo2 = __half2half2(__float2half_rd(lo)), hi2 = __half2half2(__float2half_ru(hi));
    raw_runs([&](const T (&v)[P], int c) {
      bool any = all;
      if constexpr (P == 8) {
        const __half2* h = reinterpret_cast<const __half2*>(v);
        uint32_t in = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) in |= __hge2_mask(h[i], lo2) & __hle2_mask(h[i], hi2);
        any |= in != 0;
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) any |= as_float(v[i]) >= lo && as_float(v[i]) <= hi;
      }
      if (!any) return;
      float x[P];
      widen(v, x);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float q = coord_of(x[i]);
        if (q >= c0 && q <= c1) list(which, x[i], c * P + i);
      }
    });
    sync();
  }
  // The blocks' lists together, sorted, in cand, with their running weights from `above` on in cum; returns how many, or
  // -1 if they are more than kCap.
  __device__ int arrange(int which, u64 above) {
    u64* mine = reinterpret_cast<u64*>(&sm_.w1) + which * kCap;
    int cnt[NB], n = 0;
#pragma unroll
    for (int r = 0; r < NB; ++r) cnt[r] = (int)*at(&sm_.listed[which], r);
#pragma unroll
    for (int r = 0; r < NB; ++r) n += cnt[r];
    if (n > kCap) return -1;
    // token q of the row: place q - off of the block whose list holds it; a thread's are tid, tid + TH
    constexpr int per = kCap / TH;
    u64 v[per];
#pragma unroll
    for (int e = 0; e < per; ++e) {
      int q = tid_ + e * TH, r = 0;
#pragma unroll
      for (int k = 0; k < NB - 1; ++k)
        if (r == k && q >= cnt[k]) q -= cnt[k], ++r;
      v[e] = tid_ + e * TH < n ? *at(mine + q, r) : 0;
    }
    int m = 32;
    while (m < n) m *= 2;
    // bitonic, falling: up to a distance of 16 within a warp's registers, beyond through shared memory
    for (int k = 2; k <= m; k *= 2)
      for (int j = k / 2; j; j /= 2) {
        if (j >= 32) {
          __syncthreads();
#pragma unroll
          for (int e = 0; e < per; ++e) sm_.cand[tid_ + e * TH] = v[e];
          __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < per; ++e) {
          const int q = tid_ + e * TH;
          if (e && q - lane_ >= m) break;
          const u64 y = j >= 32 ? sm_.cand[q ^ j] : __shfl_xor_sync(0xffffffffu, v[e], j);
          const bool larger = ((q & k) == 0) == ((q & j) == 0);  // this place takes the larger of the two
          if ((v[e] < y) == larger) v[e] = y;
        }
      }
    // running weights
    __syncthreads();
#pragma unroll
    for (int e = 0; e < per; ++e) sm_.cand[tid_ + e * TH] = v[e];
    if (per > 1) __syncthreads();
    u64 w[per], ws = 0;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const int q = tid_ * per + i;
      w[i] = q < n ? weight(value_of((uint32_t)((per > 1 ? sm_.cand[q] : v[i]) >> 32))) : 0;
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
    return n;
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
    if (tid_ == 0) sm_.above_n = by_count ? sm_.na[b] : 0, sm_.above_w = by_count ? 0 : sm_.wa[b];
    sync();  // what the histograms lie over is no longer read
    for (int i = tid_; i < (int)(sizeof(sm_.wd) / 4); i += TH) reinterpret_cast<uint32_t*>(&sm_.wd)[i] = 0;
    for (int i = tid_; i < (int)(sizeof(sm_.cd) / 4); i += TH) reinterpret_cast<uint32_t*>(&sm_.cd)[i] = 0;
    __syncthreads();
    uint32_t prefix = 0;
#pragma unroll 1
    for (int d = 0; d < kDigits; ++d) {
      const int shift = 24 - 8 * d;
      each([&](float x, int) {
        if (coord_of(x) != kMagic + b) return;
        const uint32_t k = key_of(x);
        if (k < floor_ || (d && (k >> (shift + 8)) != prefix)) return;
        const int g = (k >> shift) & 255;
        atomicAdd(&sm_.cd[d][g], 1u);
        if (d < kDigits - 1) sm_.wd[d].add(g, weight(x));
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
        if (d == kDigits - 1 && c) w = c * weight(value_of((prefix << 8) | g));
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
    const u64 one = weight(value_of(prefix));
    p.tie = by_count ? (uint32_t)(target - sm_.above_n) : (uint32_t)((target - p.above_w + one - 1) / one);
    sync();  // the digit histograms are read before a next descent clears them
    return p;
  }

  __device__ float logit(int i) const {  // one token's, as each() gives it
    float x;
    if constexpr (ST) {
      x = as_float(x_[i]);
    } else {
      x = as_float(reinterpret_cast<const T*>(a_.logits)[(int64_t)row_ * a_.ld + v0_ + i]);
      if (a_.allowed && !((a_.allowed[(int64_t)row_ * ((a_.vocab + 31) / 32) + ((v0_ + i) >> 5)] >> ((v0_ + i) & 31)) & 1))
        x = NAN;
    }
    return infinite_ ? (x == INFINITY ? 0.f : NAN) : x;
  }
  // Writes token and probability of tie number p.tie of key p.key, whichever block holds it.
  __device__ void locate(const Place& p, u64 total) {
    // every block's count of the key, over its threads' contiguous parts
    const int per = (n_ + TH - 1) / TH, i0 = min(n_, tid_ * per), i1 = min(n_, i0 + per);
    const float v = value_of(p.key);
    uint32_t mine = 0;
    for (int i = i0; i < i1; ++i) mine += logit(i) == v;
    uint32_t incl = mine;
    u64 none = 0;
    scan(incl, none);
    if (tid_ == TH - 1) sm_.listed[0] = incl;
    sync();
    uint32_t before = incl - mine;
    for (int r = 0; r < rank_; ++r) before += *at(&sm_.listed[0], r);
    if (before < p.tie && p.tie <= before + mine)
      for (int i = i0; i < i1; ++i)
        if (logit(i) == v && ++before == p.tie) {
          write(v0_ + i, p.key, total);
          break;
        }
  }
  __device__ void write(int32_t index, uint32_t key, u64 total) {
    a_.token[row_] = index;
    if (a_.prob) a_.prob[row_] = w_.template share<kExact>(value_of(key), total);
  }

  __device__ void draw(int k, bool use_p, float top_p, bool use_m, u64 least, float u) {
    if (k) {
      // the k-th largest of the threads' partial maxima: at least k tokens are no less
#pragma unroll
      for (int i = 0; i < 4; ++i) atomicAdd(&sm_.c1[bin_at(coord_of(infinite_ ? -INFINITY : part_max_[i]))], 1u);
      add_counts();
      int b = -1, n = -1;
      if (sm_.na[kDead] >= (uint32_t)k) {
        b = find_bin(true, k);
        gather(0, b, 0);
        n = arrange(0, 0);
      }
      if (n < 0) {  // too few maxima, or too many tokens: all counted
        sync();
        for (int i = tid_; i < kBins; i += TH) sm_.c1[i] = 0;
        if (tid_ == 0) sm_.listed[0] = 0;
        __syncthreads();
        runs([&](const float (&x)[P], int) {
#pragma unroll
          for (int i = 0; i < P; ++i) atomicAdd(&sm_.c1[bin_at(coord_of(x[i]))], 1u);
        });
        add_counts();
        if (sm_.na[kDead] <= (uint32_t)k) {
          k = 0;
        } else {
          b = find_bin(true, k);
          if (sm_.na[b + 1] <= (uint32_t)kCap) {
            gather(0, b, 0);
            n = arrange(0, 0);
          } else {
            floor_ = descend(true, b, k).key;
          }
        }
      }
      if (n >= 0) {  // the first k tokens are the first k of these
        int keep = k;
        if (use_p) keep = min(keep, reach(keep, part_of(top_p, sm_.cum[keep - 1]), 0) + 1);
        if (use_m) keep = min(keep, heavy(keep, least));
        const u64 total = sm_.cum[keep - 1];
        const int i = reach(keep, beyond(u, total), 0);
        if (rank_ == 0 && tid_ == 0) write((int32_t)~(uint32_t)sm_.cand[i], (uint32_t)(sm_.cand[i] >> 32), total);
        return;
      }
      // top-k keeps every token, or ends among too many equal ones (at floor_)
      sync();
      for (int i = tid_; i < (int)(sizeof(sm_.w1) / 16); i += TH)
        reinterpret_cast<uint4*>(&sm_)[i] = make_uint4(0, 0, 0, 0);
      if (tid_ == 0) sm_.listed[0] = 0;
      __syncthreads();
    }
    by_weight(k, use_p, top_p, use_m, least, u);
  }
  // Of `keep` sorted tokens from the first, those of at least min-p's weight (the first always).
  __device__ int heavy(int keep, u64 least) {
    if (tid_ == 0) sm_.at = keep;
    __syncthreads();
    for (int i = tid_; i < keep; i += TH)
      if (sm_.cum[i] - (i ? sm_.cum[i - 1] : 0) < least) atomicMin(&sm_.at, (uint32_t)i);
    __syncthreads();
    const int m = (int)sm_.at;
    __syncthreads();
    return max(m, 1);
  }

  // The place that target reaches in the bins' weights; with its token where its bin is not too full. list: 0 or 1.
  __device__ Place place(u64 target, int which) {
    const int b = find_bin(false, target);
    if (b != held_) {
      gather(b, b, which);
      held_n_ = arrange(which, sm_.wa[b]);
      held_ = held_n_ < 0 ? -1 : b;
    }
    if (held_ < 0) return descend(false, b, target);
    const int i = reach(held_n_, target, sm_.wa[b]);
    Place p;
    p.key = (uint32_t)(sm_.cand[i] >> 32);
    p.index = (int32_t)~(uint32_t)sm_.cand[i];
    p.above_w = sm_.cum[i];  // up to and with the token
    p.tie = 0;
    return p;
  }

  // k: top-k, whose last key is floor_, or 0.
  __device__ void by_weight(int k, bool use_p, float top_p, bool use_m, u64 least, float u) {
    u64 m_sum = 0;
    uint32_t m_key = 0xffffffffu, tokens = 0;
    const float least_logit = k ? value_of(floor_) : -INFINITY;
    // tokens of three limbs, and those that min-p may keep: t below this
    const float t_few = use_m ? fmaxf(10.0f, 40.01f - log2f(__ull2float_rn(least))) : 10.0f;
    const int few = (int)(fminf(t_few, 41.0f) * 256.0f) + kMagicBits - 2560;
    runs([&](const float (&x)[P], int) {
      uint32_t m[P];
      int bits[P];
      float c[P];
      bool rare = false;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float t = w_.t(x[i]);
        if (k && !(x[i] >= least_logit)) t = kDeadT;  // cut off
        c[i] = coord(t);
        w_.template split<kExact>(x[i], t, m[i], bits[i]);
        rare |= bits[i] < few;
        if (bits[i] >= few && c[i] < kMagic + kDead) sm_.w1.add_small(bin_at(c[i]), w_.small(m[i], bits[i]));
      }
      if (rare) {
#pragma unroll
        for (int i = 0; i < P; ++i)
          if (bits[i] < few) {
            const u64 w = w_.any(m[i], bits[i]);
            sm_.w1.add(bin_at(c[i]), w);
            if (use_m && w >= least) m_sum += w, m_key = min(m_key, key_of(x[i]));
          }
      }
      if (k) {
#pragma unroll
        for (int i = 0; i < P; ++i) tokens += c[i] < kMagic + kDead;
      }
    });
    if (use_m || k) {
      scan(tokens, m_sum);
      m_key = __reduce_min_sync(0xffffffffu, m_key);
      if (lane_ == 0) sm_.red_d[warp_] = m_key;
      __syncthreads();
      if (tid_ == TH - 1) {
        for (int i = 0; i < kWarps; ++i) m_key = min(m_key, sm_.red_d[i]);
        sm_.min_key = m_key, sm_.min_sum = m_sum, sm_.tokens = tokens;
      }
    }
    add_weights();
    uint32_t end_key = floor_;
    u64 total = sm_.wa[kDead];
    if (use_m || k) {
      m_sum = 0, m_key = 0xffffffffu, tokens = 0;
#pragma unroll
      for (int r = 0; r < NB; ++r) {
        m_sum += *at(&sm_.min_sum, r);
        m_key = min(m_key, *at(&sm_.min_key, r));
        tokens += *at(&sm_.tokens, r);
      }
      // what top-k keeps: all at or above its last key, without the ties past its last token
      if (k) total -= weight(value_of(floor_)) * (tokens - (uint32_t)k);
    }
    if (use_p) {
      const Place p = place(part_of(top_p, total), 0);
      total = p.above_w + p.tie * weight(value_of(p.key));
      end_key = p.key;
    }
    if (use_m) {
      if (m_key == 0xffffffffu) total = 1ull << kOneShift;  // min-p above one
      else if (m_key > end_key) total = m_sum;
    }
    const Place p = place(beyond(u, total), 1);
    if (p.index < 0) locate(p, total);
    else if (rank_ == 0 && tid_ == 0) write(p.index, p.key, total);
  }

  const SampleArgs& a_;
  SampleSmem<NB>& sm_;
  T* x_;
  cg::cluster_group cl_;
  const int tid_, lane_, warp_, rank_, row_;
  int v0_ = 0, n_ = 0;
  Weight w_{};
  float per_t_ = 0.f;       // bins per unit of t
  float part_max_[4];       // this thread's four partial maxima
  bool infinite_ = false;   // the largest logit is infinite
  int held_ = -1, held_n_ = 0;  // the bin whose tokens are arranged, and how many
  uint32_t floor_ = 0;  // keys below are cut off (top-k by descent)
};

// ---------------------------------------------------------------- fp16, a block a row: every value counted
// A number in fp16 has one of 65,536 patterns, so a row's tokens are counted by their pattern, in 16 bits each (128 KB):
// one shared-memory add a token instead of a weight's 40 instructions and two adds. Weights are then those of the 63,488
// numbers, w times count, added up in chunks of 64 neighbouring patterns; every place is found on the chunks' running
// sums and inside one chunk, and the row is read once more for the token's index among its equals.
// A count can pass 16 bits where more than half of the row's tokens are equal; then the counts do not add up to
// the tokens, and the row goes the other way.
constexpr int kCountFrom = 40000;  // tokens of a row above which it may be counted
constexpr int kListUpTo = 448;     // largest top-k of one that is not
constexpr int kCountThreads = 1024, kChunks = 1024, kOrdered = 993;  // 497 chunks from +inf down to 0, 496 below
struct CountSmem {
  uint32_t count[32768];   // patterns 2 i and 2 i + 1
  u64 cw[kOrdered + 1];    // weight above chunk c of the falling order
  uint32_t cn[kOrdered + 1];
  uint2 table[256];
  u64 red_w[32];
  uint32_t red_c[32];
  uint32_t tiles[kCountThreads];
  // results, written by one thread
  uint32_t chunk, bits, tie, at;
  u64 above_w;
};

class CountedRow {
 public:
  __device__ CountedRow(const SampleArgs& a, CountSmem& sm)
      : a_(a), sm_(sm), tid_(threadIdx.x), lane_(threadIdx.x & 31), warp_(threadIdx.x >> 5), row_(blockIdx.x),
        g_(reinterpret_cast<const __half*>(a.logits) + (int64_t)row_ * a.ld),
        bits_(a.allowed ? a.allowed + (int64_t)row_ * ((a.vocab + 31) / 32) : nullptr),
        wide_((reinterpret_cast<uintptr_t>(g_) & 15) == 0) {}

  // False, with nothing written, where the counts did not fit.
  __device__ bool run() {
    for (int i = tid_; i < 32768 / 4; i += kCountThreads)
      reinterpret_cast<uint4*>(sm_.count)[i] = make_uint4(0, 0, 0, 0);
    if (tid_ < 256) sm_.table[tid_] = make_uint2(kExpTable.v[tid_], __float_as_uint((float)kExpTable.v[tid_]));
    const Settings g(a_, row_);
    __syncthreads();
    uint32_t tokens = 0;
    __half2 top = __half2half2(__ushort_as_half(0xFC00));
    tokens_(&tokens, &top);
    const float2 tf = __half22float2(top);
    float mx = warp_max(fmaxf(tf.x, tf.y));
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if (lane_ == 0) sm_.red_c[warp_] = tokens, sm_.tiles[warp_] = __float_as_uint(mx);
    __syncthreads();
    mx = warp_max(__uint_as_float(sm_.tiles[lane_]));
    tokens = __reduce_add_sync(0xffffffffu, sm_.red_c[lane_]);
    __syncthreads();
    const bool none = !(mx > -INFINITY);
    if (none || g.greedy) {
      if (!none) locate(__half_as_ushort(__float2half_rn(mx)), 1, 0);
      else if (tid_ == 0) write(-1, 0, 0);
      return true;
    }
    infinite_ = mx == INFINITY;  // infinite logits share all the weight
    w_ = Weight{infinite_ ? 0.f : mx, g.kh, g.kl, sm_.table};
    if (add_counts() != tokens) return false;
    const bool use_k = g.top_k && sm_.cn[kOrdered] > (uint32_t)g.top_k;
    if (use_k) find_chunk(true, g.top_k);
    add_weights(use_k ? (int)sm_.chunk : kOrdered - 1);

    // the kept prefix, as its weight and last token's (chunk, place among the chunk's)
    u64 total = sm_.cw[kOrdered];
    Place end;
    end.key = 0;  // here: the order of the last kept pattern, larger is later; 0: everything
    bool cut = false;
    if (use_k) {
      end = find(true, g.top_k);
      total = end.above_w + end.tie * weight(end.index);
      cut = true;
    }
    if (g.use_p) {
      end = find(false, part_of(g.top_p, total));
      total = end.above_w + end.tie * weight(end.index);
      cut = true;
    }
    if (g.use_m) {
      const u64 m = heavy(g.least);  // weight of the patterns that min-p keeps; its last in sm_.bits
      if (m == 0) total = 1ull << kOneShift;
      else if (!cut || order_of(sm_.bits) < order_of(end.index)) total = m;
      __syncthreads();
    }
    const Place p = find(false, beyond(g.u, total));
    locate(p.index, p.tie, total);
    return true;
  }

 private:
  // f(8 patterns in pairs, which of them may be drawn, first token) over the row, 4 runs of 8 in flight per thread.
  template <typename F>
  __device__ __forceinline__ void runs(F f) const {
    constexpr int U = 4;
    for (int c0 = tid_; c0 * 8 < a_.vocab; c0 += U * kCountThreads) {
      uint4 v[U];
      uint32_t ok[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i0 = (c0 + k * kCountThreads) * 8;
        ok[k] = 0;
        v[k] = make_uint4(0, 0, 0, 0);
        if (i0 >= a_.vocab) continue;
        const int live = min(8, a_.vocab - i0);
        ok[k] = (bits_ ? bits_[i0 >> 5] >> (i0 & 31) : 0xFFu) & ((1u << live) - 1);
        if (wide_ && live == 8) {
          v[k] = __ldg(reinterpret_cast<const uint4*>(g_ + i0));
        } else {
          uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < live) w[i >> 1] |= (uint32_t)__half_as_ushort(g_[i0 + i]) << (16 * (i & 1));
          v[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (ok[k] == 0) continue;
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        f(w, ok[k], (c0 + k * kCountThreads) * 8);
      }
    }
  }
  __device__ __forceinline__ void add(uint32_t pattern) {
    atomicAdd(&sm_.count[pattern >> 1], (pattern & 1) ? 65536u : 1u);
  }
  // Counts the row's tokens by pattern; this thread's tokens that may be drawn, and its largest logits.
  __device__ void tokens_(uint32_t* n, __half2* top) {
    runs([&](const uint32_t (&raw)[4], uint32_t ok, int) {
      uint32_t w[4];  // -0 as 0
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = h2_as_u32(__hadd2(u32_as_h2(raw[i]), u32_as_h2(0u)));
      *n += __popc(ok);
      if (ok == 0xFFu) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          *top = __hmax2(*top, u32_as_h2(w[i]));
          add(w[i] & 0xFFFFu);
          add(w[i] >> 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((ok >> i) & 1) {
            const uint32_t p = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
            *top = __hmax2(*top, __half2half2(__ushort_as_half((uint16_t)p)));
            add(p);
          }
      }
    });
  }
  __device__ __forceinline__ uint32_t count_of(uint32_t pattern) const {
    return (sm_.count[pattern >> 1] >> (16 * (pattern & 1))) & 0xFFFFu;
  }
  // Place of a number's pattern in the falling order.
  __device__ static int order_of(uint32_t p) { return (p & 0x8000u) ? 0x7C00 + (int)(p & 0x7FFFu) : 0x7C00 - (int)p; }
  // Pattern j of ordered chunk c, in falling order.
  __device__ static uint32_t pattern_of(int c, int j) {
    return c <= 496 ? (uint32_t)((496 - c) * 64 + 63 - j) : (uint32_t)((c + 15) * 64 + j);
  }
  __device__ __forceinline__ u64 weight(uint32_t p) const {
    if (infinite_) return p == 0x7C00u ? 1ull << kOneShift : 0;
    const float x = __half2float(__ushort_as_half((uint16_t)p));
    if (!(x <= w_.mx) || !(w_.t(x) < kMaxT)) return 0;
    return w_.template value<false>(x);
  }

  // Every ordered chunk's tokens as running sums, in falling order; the tokens counted, of any pattern.
  __device__ uint32_t add_counts() {
    uint32_t counted = 0;
    for (int q = warp_; q < kChunks; q += kCountThreads / 32) {  // patterns 64 q .. 64 q + 63, two a lane
      const uint32_t c = sm_.count[q * 32 + lane_];
      const int o = q <= 496 ? 496 - q : (q >= 512 && q < 1008 ? q - 15 : -1);
      uint32_t n = __reduce_add_sync(0xffffffffu, (c & 0xFFFFu) + (c >> 16));
      counted += n;
      if (q == 496) n = __shfl_sync(0xffffffffu, c, 0) & 0xFFFFu;  // +inf; the chunk's others are NaN
      if (o >= 0 && lane_ == 0) sm_.cn[o] = n;
    }
    if (lane_ == 0) sm_.tiles[warp_] = counted;
    __syncthreads();
    counted = __reduce_add_sync(0xffffffffu, sm_.tiles[lane_]);
    uint32_t n = tid_ < kOrdered ? sm_.cn[tid_] : 0;
    u64 none = 0;
    const uint32_t n0 = n;
    scan(n, none);
    if (tid_ < kOrdered) sm_.cn[tid_] = n - n0;
    if (tid_ == kOrdered) sm_.cn[tid_] = n;
    __syncthreads();
    return counted;
  }
  // The weights of the chunks up to `last` likewise (the others as if they weighed nothing).
  __device__ void add_weights(int last) {
    for (int o = warp_; o < kOrdered; o += kCountThreads / 32) {
      u64 w = 0;
      if (o <= last && sm_.cn[o + 1] != sm_.cn[o]) {
        const uint32_t p = pattern_of(o, 0) & ~63u, c = sm_.count[(p >> 1) + lane_];
        if (o != 0 || lane_ == 0) w = (c & 0xFFFFu) * weight(p + 2 * lane_);
        if (o != 0) w += (c >> 16) * weight(p + 2 * lane_ + 1);
        // below 2^58: the warp's sum by parts of 21 bits
        const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)w & 0x1FFFFFu);
        const uint32_t b = __reduce_add_sync(0xffffffffu, (uint32_t)(w >> 21) & 0x1FFFFFu);
        const uint32_t h = __reduce_add_sync(0xffffffffu, (uint32_t)(w >> 42));
        w = a + ((u64)b << 21) + ((u64)h << 42);
      }
      if (lane_ == 0) sm_.cw[o] = w;
    }
    __syncthreads();
    uint32_t none = 0;
    u64 w = tid_ < kOrdered ? sm_.cw[tid_] : 0;
    const u64 w0 = w;
    scan(none, w);
    if (tid_ < kOrdered) sm_.cw[tid_] = w - w0;
    if (tid_ == kOrdered) sm_.cw[tid_] = w;
    __syncthreads();
  }
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
    cb = __reduce_add_sync(0xffffffffu, cb);
#pragma unroll
    for (int o = 16; o; o >>= 1) wb += __shfl_xor_sync(0xffffffffu, wb, o);
    c += cb, w += wb;
    __syncthreads();
  }

  // The chunk in which the running count or weight reaches target.
  __device__ void find_chunk(bool by_count, u64 target) {
    if (tid_ < kOrdered) {
      const u64 lo = by_count ? sm_.cn[tid_] : sm_.cw[tid_], hi = by_count ? sm_.cn[tid_ + 1] : sm_.cw[tid_ + 1];
      if (lo < target && target <= hi) sm_.chunk = tid_;
    }
    __syncthreads();
  }
  // The place where the running count or weight reaches target, which the row's does: index is the pattern here, tie its
  // token's number, above_w the weight of the patterns above.
  __device__ Place find(bool by_count, u64 target) {
    find_chunk(by_count, target);
    if (warp_ == 0) {  // two patterns a lane
      const int c = sm_.chunk;
      const uint32_t p0 = pattern_of(c, 2 * lane_), p1 = pattern_of(c, 2 * lane_ + 1);
      const bool nan = c == 0;  // the chunk of +inf: its other patterns are NaN
      const uint32_t n0 = nan && p0 != 0x7C00u ? 0 : count_of(p0), n1 = nan && p1 != 0x7C00u ? 0 : count_of(p1);
      const u64 w0 = n0 ? weight(p0) : 0, w1 = n1 ? weight(p1) : 0;
      uint32_t n = n0 + n1;
      u64 w = n0 * w0 + n1 * w1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t cu = __shfl_up_sync(0xffffffffu, n, o);
        const u64 wu = __shfl_up_sync(0xffffffffu, w, o);
        if (lane_ >= o) n += cu, w += wu;
      }
      // before p0, before p1, after p1
      const u64 wb = sm_.cw[c] + w - n0 * w0 - n1 * w1, wm = wb + n0 * w0;
      const u64 nb = sm_.cn[c] + n - n0 - n1, nm = nb + n0;
      const u64 b0 = by_count ? nb : wb, b1 = by_count ? nm : wm, b2 = by_count ? nm + n1 : wm + n1 * w1;
      if (b0 < target && target <= b1) {
        sm_.bits = p0, sm_.above_w = wb;
        sm_.tie = (uint32_t)(by_count ? target - nb : (target - wb + w0 - 1) / w0);
      } else if (b1 < target && target <= b2) {
        sm_.bits = p1, sm_.above_w = wm;
        sm_.tie = (uint32_t)(by_count ? target - nm : (target - wm + w1 - 1) / w1);
      }
    }
    __syncthreads();
    Place p;
    p.index = (int32_t)sm_.bits;
    p.tie = sm_.tie;
    p.above_w = sm_.above_w;
    p.key = 1;
    __syncthreads();
    return p;
  }

  // Weight of the tokens of at least `least`, 0 if there are none; sm_.bits: the last pattern of that weight.
  __device__ u64 heavy(u64 least) {
    if (tid_ == 0) sm_.chunk = 0, sm_.above_w = 0;
    __syncthreads();
    // the last chunk whose first pattern weighs enough (those from the largest logit's chunk on)
    const int first = order_chunk();
    if (tid_ < kOrdered && tid_ > first && weight(pattern_of(tid_, 0)) >= least) atomicMax(&sm_.chunk, (uint32_t)tid_);
    __syncthreads();
    if (warp_ == 0) {
      const int c = max((int)sm_.chunk, first);
      const uint32_t p0 = pattern_of(c, 2 * lane_), p1 = pattern_of(c, 2 * lane_ + 1);
      const bool nan = c == 0;
      const u64 w0 = nan && p0 != 0x7C00u ? 0 : weight(p0), w1 = nan && p1 != 0x7C00u ? 0 : weight(p1);
      const bool k0 = w0 >= least, k1 = w1 >= least;
      u64 w = (k0 ? count_of(p0) * w0 : 0) + (k1 ? count_of(p1) * w1 : 0);
#pragma unroll
      for (int k = 16; k; k >>= 1) w += __shfl_xor_sync(0xffffffffu, w, k);
      const uint32_t a = __ballot_sync(0xffffffffu, k0 || k1);
      if (lane_ == 0) {
        sm_.above_w = a ? sm_.cw[c] + w : 0;
        if (!a) sm_.bits = 0;
      }
      if (a && lane_ == 31 - __clz(a)) sm_.bits = k1 ? p1 : p0;
    }
    __syncthreads();
    const u64 w = sm_.above_w;
    __syncthreads();
    return w;
  }
  __device__ int order_chunk() const {  // the largest logit's chunk
    if (infinite_) return 0;
    const uint32_t p = __half_as_ushort(__float2half_rn(w_.mx));
    return (p & 0x8000u) ? (int)(p >> 6) - 15 : 496 - (int)(p >> 6);
  }

  // Writes the tie-th token (from 1) of a pattern, found by tiles of 256 tokens.
  __device__ void locate(uint32_t pattern, uint32_t tie, u64 total) {
    // a warp's run of 256 tokens is a tile; their tokens of the pattern
    const int n_tiles = (a_.vocab + 255) / 256;
    for (int i = tid_; i < kCountThreads; i += kCountThreads) sm_.tiles[i] = 0;
    __syncthreads();
    const __half2 wanted = u32_as_h2(pattern * 0x10001u);
    runs([&](const uint32_t (&v)[4], uint32_t ok, int i0) {
      uint32_t eq[4];  // all ones in the halves that are equal
#pragma unroll
      for (int i = 0; i < 4; ++i) eq[i] = __heq2_mask(u32_as_h2(v[i]), wanted);
      if (!(eq[0] | eq[1] | eq[2] | eq[3])) return;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m |= (eq[i] & 1u) << (2 * i) | (eq[i] >> 31) << (2 * i + 1);
      m &= ok;
      if (m) atomicAdd(&sm_.tiles[i0 >> 8], __popc(m));
    });
    __syncthreads();
    uint32_t n = tid_ < n_tiles ? sm_.tiles[tid_] : 0;
    const uint32_t mine = n;
    u64 none = 0;
    scan(n, none);
    if (n - mine < tie && tie <= n) sm_.at = tid_, sm_.tie = tie - (n - mine);
    __syncthreads();
    if (warp_ == 0) {
      const int i0 = (int)sm_.at * 256 + lane_ * 8;
      uint32_t m = 0;
      for (int i = 0; i < 8; ++i) {
        if (i0 + i >= a_.vocab) break;
        if (bits_ && !((bits_[(i0 + i) >> 5] >> ((i0 + i) & 31)) & 1)) continue;
        const uint32_t p = __half_as_ushort(g_[i0 + i]);
        m |= (uint32_t)((p == 0x8000u ? 0u : p) == pattern) << i;
      }
      uint32_t c = __popc(m);
      const uint32_t own = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, c, o);
        if (lane_ >= o) c += u;
      }
      uint32_t left = sm_.tie - (c - own);  // the wanted one's number among the lane's, if it is there
      if (c - own < sm_.tie && sm_.tie <= c) {
        while (--left) m &= m - 1;
        write(i0 + __ffs(m) - 1, pattern, total);
      }
    }
  }
  // total 0: the first largest logit, for itself
  __device__ void write(int32_t index, uint32_t pattern, u64 total) {
    a_.token[row_] = index;
    if (!a_.prob) return;
    if (index < 0) a_.prob[row_] = __int_as_float(0x7fc00000);
    else if (total == 0) a_.prob[row_] = 1.0f;
    else a_.prob[row_] = w_.template share<false>(infinite_ ? 0.f : __half2float(__ushort_as_half((uint16_t)pattern)), total);
  }

  const SampleArgs& a_;
  CountSmem& sm_;
  const int tid_, lane_, warp_, row_;
  const __half* g_;
  const uint32_t* bits_;
  const bool wide_;
  Weight w_{};
  bool infinite_ = false;
};

__global__ void __launch_bounds__(kCountThreads, 1) sample_counted_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  // a row with a small top-k needs no count, since the partial maxima bring it down to a short list: 256 rows of 128,256,
  // 51 us counted, listed 34 at k = 50, 43 at 200, 50 at 450, 55 at 512 (a longer sort), 74 at 1,024; others alike
  const int k = a.top_k ? a.top_k[blockIdx.x] : 0;
  if ((k <= 0 || k > kListUpTo) && CountedRow(a, *reinterpret_cast<CountSmem*>(smem_raw)).run()) return;
  __syncthreads();
  Sampler<__half, 1, kCountThreads, false>(a, *reinterpret_cast<SampleSmem<1>*>(smem_raw), nullptr).run();
}

template <typename T, int NB, int TH, bool ST>
__global__ void __launch_bounds__(TH, ST ? 1 : 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SampleSmem<NB>& sm = *reinterpret_cast<SampleSmem<NB>*>(smem_raw);
  T* x = reinterpret_cast<T*>(smem_raw + (sizeof(SampleSmem<NB>) + 15) / 16 * 16);
  Sampler<T, NB, TH, ST>(a, sm, x).run();
}

template <typename T, int NB, int TH, bool ST>
cudaError_t launch_sample_th(cudaStream_t s, const SampleArgs& a, size_t slice) {
  const size_t smem = (sizeof(SampleSmem<NB>) + 15) / 16 * 16 + (ST ? slice : 0);
  cudaError_t e =
      cudaFuncSetAttribute(sample_kernel<T, NB, TH, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, NB, TH, ST>, a);
}
template <typename T, int NB>
cudaError_t launch_sample_nb(cudaStream_t s, const SampleArgs& a, size_t slice) {
  // a slice of more than 8 tokens a thread: twice the threads
  return slice / sizeof(T) > 512 * 8 ? launch_sample_th<T, NB, 1024, true>(s, a, slice)
                                      : launch_sample_th<T, NB, 512, true>(s, a, slice);
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
  if constexpr (sizeof(T) == 2) {
    // Counting clears and adds up 65,536 counts a row, however short, and has an SM a row, so it is for long rows and
    // many. fp16 without cuts / with top-p, us, counted and by bins: 128,256 tokens, 20 rows 33 and 27 / 34 and 37, 40 rows
    // 33 and 39 / 34 and 49, 256 rows 65 and 133 / 68 and 158; 50,000 tokens, 40 rows 25 and 24 / 27 and 29, 256 rows 50 and
    // 60 / 53 and 72; 32,000 tokens, 40 rows 23 and 18 / 24 and 23, 256 rows 45 and 40 / 48 and 51; 1,000 tokens,
    // 40 rows 18 and 8 / 20 and 11, 256 rows 34 and 11 / 37 and 17.
    if (a.vocab > kCountFrom && a.vocab <= kMaxSlice && (int64_t)a.rows * 4 > n_sm) {
      constexpr int smem = (int)std::max(sizeof(CountSmem), sizeof(SampleSmem<1>));
      e = cudaFuncSetAttribute(sample_counted_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      return launch_kernel(Launch{s, false, nullptr}, sample_counted_kernel, dim3(a.rows), dim3(kCountThreads), smem, a);
    }
  }
  // a row or more for every SM: a block a row
  if (a.rows >= n_sm && a.vocab <= kMaxSlice) return launch_sample_th<T, 1, 512, false>(s, a, 0);
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
