// The next token of every row of logits from a given uniform number (nld_sample).
//
// With x the row's logits and T its temperature, w_i = exp((x_i - max x) / T).  In the order of
// falling logits, equal ones by index: top-k keeps the first k tokens; top-p the tokens of these
// before which less than p of their mass lies (one at least); min-p the tokens of these with
// w_i >= min_p.  The sampled token is the first kept one, by index, up to and with which more than
// u of the kept mass lies.
//
// A cluster of up to 8 CTAs takes a row.  Each reads its slice once, into shared memory, and every
// later pass runs on that copy, so a logit crosses HBM once.
//
// The kept tokens are those whose logit exceeds a border value and the first few, by index, that
// equal it.  A border is found by histograms of counts (top-k) or masses (top-p), of kBins bins
// in the order of falling logits: the first over equal steps of (max x - x) / T, kOctave per
// halving of the weight; the next over the order-preserving keys inside the border's bin, until
// that bin is one key (three levels for fp32, two for bf16, whatever the values).  Every
// CTA counts its slice; one cluster barrier later each of them finds the bin from all CTAs'
// range sums and that range's bins over distributed shared memory.
//
// Adding to shared memory is what a histogram costs (18 cycles a warp), so the first levels add less:
//   - for a small k, of each thread's largest logit alone: the k-th of those bounds the border from below, and
//     the tokens from there on are few;
//   - for p, one 32-bit number a token, its weight over that of its bin's start, to 2^-15: two or three bins that
//     must hold the border.  The next pass takes the exact total and the exact mass over those bins in
//     registers and counts the tokens inside exactly.  If the border is not there after all, the exact first
//     level follows.
// Where at most kList tokens are left (most calls with top-k, and peaked rows), one CTA ranks them against one
// another instead, and neither further levels nor another pass over the row follow.
//
// Masses are sums of 64-bit fixed-point weights (2^44 at the row's largest logit; up to 2^19
// tokens fit): their sums do not depend on the order of addition, so neither do the borders or the
// token.  In the histograms a weight is three 15-bit limbs, each with a 32-bit counter of its own
// (a slice has at most 2^16 tokens), because shared memory adds 32-bit integers natively.
#include <atomic>
#include <cstddef>

#include "common.cuh"

namespace nld {

namespace {

constexpr int kMaxWarps = 16;       // of a CTA: 16, or 8 (see the launcher)
constexpr int kMaxS = 8;            // CTAs of a row
constexpr int kBins = 1024;
constexpr int kRanges = 32;         // of 32 bins
constexpr int kOctave = 20;         // bins per halving: the last one starts at 2^-51, no weight
constexpr int kList = 256;          // tokens ranked against one another
constexpr float kFltMax = 3.402823466e38f;
constexpr double kOne = 17592186044416.0;   // 2^44: the weight of the largest logit

typedef unsigned long long u64;

// Keys in the order of the values, of as many bits as the type has; -inf has the key kInf.  (A NaN's key
// is over that of +inf or under that of -inf.)
template <typename T>
struct Key;
template <>
struct Key<float> {
  static constexpr int n = 4;   // logits per 16 bytes
  typedef uint4 Quad;           // 4 logits
  static constexpr uint32_t kInf = 0x007fffffu;
  static NLD_DEV uint32_t of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);   // -0 as +0
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  }
  static NLD_DEV float value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }
  static NLD_DEV void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static NLD_DEV float most(const uint4& v) {   // the largest; NaN does not count
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
};
template <>
struct Key<__nv_bfloat16> {
  static constexpr int n = 8;
  typedef uint2 Quad;
  static constexpr uint32_t kInf = 0x007fu;
  static NLD_DEV uint32_t of(float x) { return Key<float>::of(x) >> 16; }
  static NLD_DEV float value(uint32_t k) {
    return __uint_as_float((k & 0x8000u) ? (k ^ 0x8000u) << 16 : (k ^ 0xffffu) << 16);
  }
  static NLD_DEV void unpack(const uint2& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  static NLD_DEV float most(const uint4& v) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 m = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};

// For Weigh::biased: 1.5 2^52, the polynomial from its highest coefficient on, 2^52.  (In constant memory, an
// operand that costs no instruction: as literals they were two moves each.)
__constant__ double kExp[8] = {6755399441055744.0,     1.2716085030349987e-09, 1.4676444621898709e-07, 1.355080777749983e-05,
                               0.000938384792486206, 0.043321698784996608,   1.0,                    4503599627370496.0};

__device__ const double kTab[16] = {17592186044416.0, 18371058661769.06, 19184414915921.48, 20033781527906.22,
                                    20920752812471.082, 21846993670708.133, 22814242715178.152, 23824315533396.16,
                                    24879108095803.8, 25980600314625.527, 27130859760288.855, 28332045542384.562,
                                    29586412362451.676, 30896314746194.61, 32264211463076.527, 33692670141584.85};   // 2^(44 + j / 16)

// Weights of a row's logits.
struct Weigh {
  float top, half_top;   // the largest logit; FLT_MAX for +inf (then `low` leaves only those of +inf)
  float low;             // logits under it have no weight (NaN compares as one of them)
  float steps, more;     // their product: bins of the first level per unit of (max x - x) / 2
  double top_d, inv_t, s16;
  const double* tab;     // 2^(44 + j / 16), j = 0..15, j 2^16 off the high words (k's low bits add it back)
  NLD_DEV void init(float top_, float temperature, const double* tab_) {
    top = fminf(top_, kFltMax);
    half_top = 0.5f * top;   // halves: the difference of two finite logits may exceed fp32
    top_d = static_cast<double>(top);
    inv_t = 1.0 / static_cast<double>(temperature);
    s16 = inv_t * 23.083120654223414;   // 16 log2(e)
    // 50 halvings down (fp32 rounding leaves it under 120); 2^-45 rounds to nothing
    low = top_ > kFltMax ? top_ : fmaxf(static_cast<float>(top_d - 34.657 * static_cast<double>(temperature)), -kFltMax);
    const double per = inv_t * (2.0 * 1.4426950408889634 * kOctave);
    steps = static_cast<float>(fmin(per, 1e38));
    more = per > 1e38 ? static_cast<float>(per * 1e-38) : 1.f;
    tab = tab_;
  }
  // Bin of the first level of a logit not under `low`: not falling as x falls.
  NLD_DEV float depth(float x) const {   // in bins
    float d = (half_top - 0.5f * fminf(x, kFltMax)) * steps;
    if (more != 1.f) d *= more;
    return fminf(d, static_cast<float>(kBins - 1));
  }
  NLD_DEV int bin(float x) const { return static_cast<int>(depth(x)); }
  // exp((x - top) / T) 2^44 + 2^52, rounded to a whole number, as the bits of the double (kBias + the
  // weight); kBias where !in, or where x is under `low` and not in.  With y = 16 log2(e) (x - top) / T = k + r,
  // |r| <= 1/2: 2^(y / 16) = 2^(k / 16) p(r), p the Chebyshev interpolant of degree 5 of 2^(r / 16) with p(0)
  // set to 1: within 2^-46 of it.  Adding 1.5 2^52 rounds y, adding 2^52 the weight.
  static constexpr u64 kBias = 0x4330000000000000ull;
  NLD_DEV u64 biased(float x, bool in) const {
    double p;
    const double scaled = parts(fminf(fmaxf(x, low), kFltMax), in, p);
    return static_cast<u64>(__double_as_longlong(fma(scaled, p, kExp[7])));
  }
  // The same for every logit of a row with plain(): what is under `low` counts as `low`, which has no weight.
  NLD_DEV u64 biased(float x) const {
    double p;
    const double scaled = parts(fmaxf(x, low), true, p);
    return static_cast<u64>(__double_as_longlong(fma(scaled, p, kExp[7])));
  }
  NLD_DEV bool plain() const { return top < kFltMax && fixed(low) == 0; }
  NLD_DEV double parts(float x, bool in, double& p) const {
    const double d = static_cast<double>(x) - top_d;
    const double t = fma(d, s16, kExp[0]);
    const double r = fma(d, s16, kExp[0] - t);
    const int k = __double2loint(t);
    p = fma(r, kExp[1], kExp[2]);
    p = fma(r, p, kExp[3]);
    p = fma(r, p, kExp[4]);
    p = fma(r, p, kExp[5]);
    p = fma(r, p, kExp[6]);
    const double m = tab[k & 15];
    const int hi = __double2hiint(m) + (k << 16);
    return __hiloint2double(in ? hi : 0, __double2loint(m));
  }
  NLD_DEV u64 fixed(float x) const { return biased(x, true) - kBias; }
};
// The same out of line, for code that runs once: a call that samples few logits is bound by fetching its
// instructions.
__device__ __noinline__ u64 fixed_weight(const Weigh& w, float x) { return w.fixed(x); }
__device__ __noinline__ double real_weight(const Weigh& w, float x) {   // not rounded to a whole number
  double p;
  const double scaled = w.parts(fminf(fmaxf(x, w.low), kFltMax), true, p);
  return scaled * p;
}

NLD_DEV float exp2_hw(float x) {   // relative error about 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename V>
NLD_DEV V warp_sum(V v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// Sum over the lanes up to and with this one.
template <typename V>
NLD_DEV V warp_scan(V v) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const V o = __shfl_up_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) >= off) v += o;
  }
  return v;
}
// Sum over the threads before this one, and over all.  `red` holds an entry a warp; callable again at
// once.
template <typename V>
__device__ __noinline__ V block_scan(V v, V* red, V& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const V inc = warp_scan(v);
  __syncthreads();
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  const V w = lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : V(0);
  const V before = warp_sum(lane < warp ? w : V(0));
  total = warp_sum(w);
  return before + inc - v;
}

NLD_DEV u64 ld_dsmem_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
NLD_DEV uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

NLD_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
NLD_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
NLD_DEV void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
NLD_DEV void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// What a CTA's peers read, and its own scratch.
struct Shared {
  u64 part_mass[kMaxWarps];     // kept mass over the border, ties at it: of each warp's part of the slice
  int part_ties[kMaxWarps];
  double tab[16];
  Weigh weigh;
  u64 red_m[kMaxWarps], red_n[kMaxWarps];
  int red_c[kMaxWarps];
  uint32_t top;                 // the slice's largest key
  int top_at;                   // the lowest index of the row's largest logit in the slice
  int listed;                   // tokens of `list` (more: not all are in it)
  int found_at;                 // warp 0's findings
  uint32_t key_lo, key_hi;
  u64 found_before, found_with, found_total;
  int found_count;
  u64 sum_total, sum_above;     // of the slice: mass, and that over the bins that must hold the border
  int sum_count;                // tokens in and over those bins
  int at_part, done;            // the sampled token's part, and what lies before that part
  u64 at_before, total;
  long long at_ties;
  double target;
  // from here on only where there is a border to find
  u64 range[2][kRanges];        // [buffer]: sums over 32 bins
  u64 gather[3][kMaxS][32];     // of the CTAs of the row: their range sums, their sums of one range's bins
  u64 sums[kMaxS][3];           // their sum_total, sum_above, sum_count
  u64 list[kList];              // key, then the index's complement
  union {
    uint32_t hist[2][3][kBins];        // [buffer][limb][bin]; counts use limb 0
    struct {
      u64 all[kList], weight[kList];   // rank 0, after the searches: the lists of all CTAs, the tokens' weights
    };
  };
};
constexpr size_t kHeadFull = (sizeof(Shared) + 15) / 16 * 16;
constexpr size_t kHeadPlain = (offsetof(Shared, range) + 15) / 16 * 16;

// One row's slice: the 16-byte vectors of it, in shared memory or (slices over the shared memory)
// straight from global memory; -inf outside the row.
template <typename T, bool kStaged>
struct Slice {
  static constexpr int n = Key<T>::n;
  const uint4* staged;
  const T* row;
  long long first;    // index of the slice's first logit (a 16-byte boundary; before the row's start by up to n - 1)
  int vocab;
  int whole0, whole1;   // vectors that lie in the row
  NLD_DEV bool whole(int v) const { return v >= whole0 && v < whole1; }
  NLD_DEV const uint4* vector(int v) const { return reinterpret_cast<const uint4*>(row + (first + static_cast<long long>(v) * n)); }
  __device__ __noinline__ uint4 ragged(int v) const {   // a vector at the row's ends
    const long long i0 = first + static_cast<long long>(v) * n;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (n == 4) {
        w[i] = i0 + i >= 0 && i0 + i < vocab ? reinterpret_cast<const uint32_t*>(row)[i0 + i] : 0xff800000u;
      } else {
        const long long e = i0 + 2 * i;
        const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
        const uint32_t lo = e >= 0 && e < vocab ? r[e] : 0xff80u, hi = e + 1 >= 0 && e + 1 < vocab ? r[e + 1] : 0xff80u;
        w[i] = lo | (hi << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  NLD_DEV void get(int q, float (&x)[4]) const {   // the 4 logits of quad q
    typedef typename Key<T>::Quad Quad;
    constexpr int per = n / 4;
    if constexpr (kStaged) {
      Key<T>::unpack(reinterpret_cast<const Quad*>(staged)[q], x);
    } else if (whole(q / per)) {
      Key<T>::unpack(__ldg(reinterpret_cast<const Quad*>(row + (first + static_cast<long long>(q) * 4))), x);
    } else {
      const uint4 v = ragged(q / per);
      Key<T>::unpack(reinterpret_cast<const Quad*>(&v)[per == 1 ? 0 : q % per], x);
    }
  }
};

template <typename T, bool kStaged, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 1024 / (32 * kWarps)) sample_kernel(const SampleArgs a) {
  constexpr int kThreads = 32 * kWarps;
  using K = Key<T>;
  constexpr int n = K::n;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint4* const stage = reinterpret_cast<uint4*>(smem + a.head);
  const int S = a.S, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % S;
  const size_t row = blockIdx.x / S;
  Slice<T, kStaged> slice;
  slice.staged = stage;
  slice.row = static_cast<const T*>(a.logits) + row * a.ld;
  slice.vocab = a.vocab;
  // the row's vectors start at the 16-byte boundary at or before it; warp w of the slice has a.part of them
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(slice.row) % 16 / sizeof(T));
  slice.first = static_cast<long long>(rank) * (a.part * kWarps * n) - skew;
  slice.whole0 = slice.first < 0 ? 1 : 0;
  slice.whole1 = max(slice.whole0, static_cast<int>(max(-1LL, min(static_cast<long long>(a.part) * kWarps, (a.vocab - slice.first) / n))));
  const int v0 = warp * a.part, v1 = v0 + a.part;
  const int q0 = v0 * (n / 4), q1 = v1 * (n / 4);   // the same in quads of logits

  // a word of CTA q's Shared, at the place of `p` in this one's
  auto peer64 = [&](const void* p, int q) -> u64 {
    return S == 1 ? *static_cast<const volatile u64*>(p) : ld_dsmem_u64(dsmem_addr(smem_u32(p), q));
  };
  auto peer32 = [&](const void* p, int q) -> uint32_t {
    return S == 1 ? *static_cast<const volatile uint32_t*>(p) : ld_dsmem_u32(dsmem_addr(smem_u32(p), q));
  };
  auto row_sync = [&]() {
    if (S == 1) __syncthreads();
    else cluster_sync();
  };

  const float temperature = a.temperature ? a.temperature[row] : 1.f;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.f;
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  const float uf = a.u[row];
  if (tid < 16) sh.tab[tid] = __hiloint2double(__double2hiint(kTab[tid]) - (tid << 16), __double2loint(kTab[tid]));
  if (tid == 0) {
    sh.listed = 0;
    sh.top_at = 0x7fffffff;
  }
  const bool by_k = k > 0 && k < a.vocab, by_p = p < 1.f;
  auto clear = [&](int buffer) {
    for (int i = tid; i < 3 * kBins / 4; i += kThreads) reinterpret_cast<uint4*>(&sh.hist[buffer][0][0])[i] = make_uint4(0, 0, 0, 0);
  };
  if (by_k || by_p) clear(0);

  // the largest logit
  float big = -INFINITY;   // of this thread's
  {
    const int w0 = max(v0, slice.whole0), w1 = min(v1, slice.whole1);
    if constexpr (kStaged) {   // all of the slice in flight; a thread reads back what it copied itself
      uint4* const to = stage;
      for (int v = w0 + lane; v < w1; v += 32) cp_async16(to + v, slice.vector(v));
      cp_async_wait();
      for (int v = w0 + lane; v < w1; v += 32) big = fmaxf(big, K::most(to[v]));
    } else {
#pragma unroll 4
      for (int v = w0 + lane; v < w1; v += 32) big = fmaxf(big, K::most(__ldg(slice.vector(v))));
    }
    if (!slice.whole(0) || !slice.whole(kWarps * a.part - 1))   // a row's ends
      for (int v = v0 + lane; v < v1; v += 32)
        if (!slice.whole(v)) {
          const uint4 got = slice.ragged(v);
          if constexpr (kStaged) stage[v] = got;
          big = fmaxf(big, K::most(got));
        }
    const uint32_t key = __reduce_max_sync(0xffffffffu, K::of(big));
    if (lane == 0) sh.red_c[warp] = static_cast<int>(key);
    __syncthreads();
    if (warp == 0) {
      const uint32_t all = __reduce_max_sync(0xffffffffu, lane < kWarps ? static_cast<uint32_t>(sh.red_c[lane]) : 0u);
      if (lane == 0) sh.top = all;
    }
  }
  row_sync();
  const uint32_t top_key = __reduce_max_sync(0xffffffffu, lane < S ? peer32(&sh.top, lane) : 0u);
  if (top_key == K::kInf || !(temperature > 0.f) || k == 1 || p <= 0.f) {   // (the same for the whole cluster)
    if (top_key != K::kInf) {   // the likeliest token alone: the lowest index with the largest logit
      const float top = K::value(top_key);
      for (int q = q0 + lane; q < q1; q += 32) {
        float x[4];
        slice.get(q, x);
        const int at = x[0] == top ? 0 : x[1] == top ? 1 : x[2] == top ? 2 : x[3] == top ? 3 : -1;
        if (at >= 0) {
          atomicMin(&sh.top_at, static_cast<int>(slice.first + static_cast<long long>(q) * 4 + at));
          break;   // this thread's later ones have higher indexes
        }
      }
    }
    row_sync();
    if (rank == 0 && warp == 0) {
      const int at = __reduce_min_sync(0xffffffffu, lane < S ? static_cast<int>(peer32(&sh.top_at, lane)) : 0x7fffffff);
      if (lane == 0) {
        a.tokens[row] = top_key == K::kInf ? -1 : at;
        if (a.prob) a.prob[row] = top_key == K::kInf ? 0.f : 1.f;
      }
    }
    row_sync();   // peers' shared memory may still be read
    return;
  }
  if (tid == 0) sh.weigh.init(K::value(top_key), temperature, sh.tab);
  __syncthreads();
  Weigh weigh = sh.weigh;
  weigh.tab = sh.tab;   // (known to be shared memory)
  const double u = uf > 0.f ? static_cast<double>(fminf(uf, 0.99999994f)) : 0.0;
  const u64 least = mp > 0.f ? static_cast<u64>(ceil(static_cast<double>(fminf(mp, 1.f)) * kOne)) : 0;

  // ------------------------------------------------------------------ the border --
  // kept: keys over `border`, and the first `ties` tokens at it
  uint32_t border = K::kInf;
  long long ties = a.vocab;
  auto over_border = [&]() {   // logits from here on are over the border and have a weight
    return border >= top_key ? NAN : fmaxf(weigh.low, K::value(border + 1));   // (NaN: none are)
  };
  // What is searched for, by number first, then by mass among the kept: kMaxima, kCount or kBracketing, kBracketed,
  // kMass are first levels of it
  enum { kMaxima, kCount, kBracketing, kBracketed, kMass };
  int kind = !by_k ? kBracketing : k <= kList - 16 ? kMaxima : kCount;
  int level = 0, buf = 0;
  u64 before = 0, rest = 0, rest_w = 0;   // over the bin; mass of the ties at the top-k border, and of one of them
  double limit = by_k ? k : p;            // first levels by mass: a share of the total
  uint32_t lo = 0, hi = 0;                // keys of the bin (levels 1 and up, and kBracketed)
  u64 above = 0;                          // kBracketed: mass of this thread's tokens over above_x
  float above_x = INFINITY;
  while (by_k || by_p) {
    // One level: tokens over the border (level 0) or with keys lo..hi, in steps of 2^shift; their numbers or masses
    // by bin, and the bin with which the sum reaches the limit.
    const bool mass = kind >= kBracketing, by_key = level > 0 || kind == kBracketed;
    uint32_t(*h)[kBins] = sh.hist[buf];
    const int shift = by_key ? max(0, 22 - __clz(hi - lo)) : 0;   // (hi - lo) >> shift < 2^10
    const float from = level == 0 ? over_border() : K::value(lo), to = by_key ? K::value(hi) : INFINITY;
    auto add = [&](int bin, u64 w) {
      uint32_t* const at = &h[0][0] + bin;
      const uint32_t w2 = static_cast<uint32_t>(w >> 30), w1 = static_cast<uint32_t>(w >> 15) & 0x7fffu;
      atomicAdd(at, static_cast<uint32_t>(w) & 0x7fffu);
      if (w1) atomicAdd(at + kBins, w1);
      if (w2) atomicAdd(at + 2 * kBins, w2);
    };
    if (level == 0 && kind == kMaxima) {
      if (big >= from) atomicAdd(&h[0][weigh.bin(big)], 1u);
    } else if (level == 0 && kind == kBracketing) {
      for (int q = q0 + lane; q < q1; q += 32) {
        float x[4];
        slice.get(q, x);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x[e] >= from) {
            const float d = weigh.depth(x[e]);
            const int b = static_cast<int>(d);
            atomicAdd(&h[0][b], __float2uint_rn(exp2_hw(fmaf(static_cast<float>(b) - d, 1.f / kOctave, 15.f))));
          }
      }
    } else if (level == 0 && kind == kBracketed) {
      const float from_lo = K::value(lo);
      u64 all = 0;
      int count = 0;
      above = 0;
      above_x = to;
      for (int q = q0 + lane; q < q1; q += 32) {
        float x[4];
        slice.get(q, x);
        if (!(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= from)) continue;
        u64 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = weigh.biased(x[e], x[e] >= from) - Weigh::kBias;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          all += w[e];
          if (x[e] > to) above += w[e];
          if (x[e] >= from_lo) {
            ++count;
            if (x[e] <= to) add(static_cast<int>((hi - K::of(x[e])) >> shift), w[e]);
          }
        }
      }
      const u64 s0 = warp_sum(all), s1 = warp_sum(above);
      const int s2 = __reduce_add_sync(0xffffffffu, count);
      if (lane == 0) {
        sh.red_m[warp] = s0;
        sh.red_n[warp] = s1;
        sh.red_c[warp] = s2;
      }
    } else {
      for (int q = q0 + lane; q < q1; q += 32) {
        float x[4];
        slice.get(q, x);
        bool in[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) in[e] = x[e] >= from && x[e] <= to;
        if (!(in[0] || in[1] || in[2] || in[3])) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!in[e]) continue;
          const int bin = by_key ? static_cast<int>((hi - K::of(x[e])) >> shift) : weigh.bin(x[e]);
          if (mass) add(bin, fixed_weight(sh.weigh, x[e]));
          else atomicAdd(&h[0][bin], 1u);
        }
      }
    }
    __syncthreads();
    const bool bracketing = level == 0 && kind == kBracketing;
    // a bin's sum (counts: the other limbs are 0; bracketing: of the weights to 2^-15, 2^43 for the largest logit's)
    auto bin_sum = [&](uint32_t w0, uint32_t w1, uint32_t w2, int b) -> u64 {
      if (bracketing) {
        const int o = b / kOctave;
        return (static_cast<u64>(w0) * __float2uint_rn(exp2f(28.f - static_cast<float>(b - o * kOctave) * (1.f / kOctave)))) >> o;
      }
      return w0 + (static_cast<u64>(w1) << 15) + (static_cast<u64>(w2) << 30);
    };
#pragma unroll 1
    for (int r = warp; r < kRanges; r += kWarps) {
      const int b = r * 32 + lane;
      const u64 s = warp_sum(bin_sum(h[0][b], h[1][b], h[2][b], b));
      if (lane == 0) sh.range[buf][r] = s;
    }
    if (warp == 0 && level == 0 && kind == kBracketed) {
      const u64 s0 = warp_sum(lane < kWarps ? sh.red_m[lane] : 0), s1 = warp_sum(lane < kWarps ? sh.red_n[lane] : 0);
      const int s2 = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.red_c[lane] : 0);
      if (lane == 0) {
        sh.sum_total = s0;
        sh.sum_above = s1;
        sh.sum_count = s2;
      }
    }
    row_sync();
    // the other buffer was last read before this barrier
    clear(buf ^ 1);
    // The row's sums, in two steps: warp q fetches CTA q's range sums, then its bins of the range with the border (a
    // warp that fetched all of them waited 4 us: a fetch is 0.2 us and the next one came after its use).
    auto of_all = [&](const u64(*g)[32]) -> u64 {
      u64 v[kMaxS], sum = 0;
#pragma unroll
      for (int q = 0; q < kMaxS; ++q) v[q] = g[min(q, S - 1)][lane];   // (all fetched before the first is used)
#pragma unroll
      for (int q = 0; q < kMaxS; ++q) sum += q < S ? v[q] : 0;
      return sum;
    };
    if (warp < S) {
      sh.gather[0][warp][lane] = peer64(&sh.range[buf][lane], warp);
      if (level == 0 && kind == kBracketed && lane < 3)
        sh.sums[warp][lane] = lane == 0 ? peer64(&sh.sum_total, warp) : lane == 1 ? peer64(&sh.sum_above, warp) : peer32(&sh.sum_count, warp);
    }
    __syncthreads();
    const int sides = bracketing ? 2 : 1;
    if (warp < max(S, 2)) {
      const u64 inc = warp_scan(of_all(sh.gather[0]));
      u64 total = __shfl_sync(0xffffffffu, inc, 31);
      u64 start = before;   // what lies before the bins
      int count = 0;
      double reach = limit;
      if (level == 0 && kind == kBracketed) {
        total = start = 0;
#pragma unroll 1
        for (int q = 0; q < S; ++q) {
          total += sh.sums[q][0];
          start += sh.sums[q][1];
          count += static_cast<int>(sh.sums[q][2]);
        }
      }
      total += bracketing ? 0 : rest;
      if (level == 0 && mass && !bracketing) reach *= static_cast<double>(total);
      if (bracketing) reach *= static_cast<double>(total) + 0.5 * static_cast<double>(rest);
      // the bin with which the sum reaches the limit; bracketing: the first that may be it (side 0), and the first that is
      // surely at it or behind (a bin's sum is off by 2^-14 of it at most)
      auto reached = [&](u64 c, int side) {
        const double d = static_cast<double>(start + c);
        return (bracketing ? d * (side == 0 ? 1.0 + 0x1p-13 : 1.0 - 0x1p-13) : d) >= reach;
      };
      int r[2];
#pragma unroll
      for (int side = 0; side < 2; ++side) r[side] = __ffs(__ballot_sync(0xffffffffu, reached(inc, side))) - 1;
      if (warp < S)
#pragma unroll 1
        for (int side = 0; side < sides; ++side)
          if (r[side] >= 0) {
            const int b = r[side] * 32 + lane;
            const uint32_t w0 = peer32(&h[0][b], warp), w1 = bracketing ? 0 : peer32(&h[1][b], warp), w2 = bracketing ? 0 : peer32(&h[2][b], warp);
            sh.gather[1 + side][warp][lane] = bin_sum(w0, w1, w2, b);
          }
      if (S == 1) __syncwarp();
      named_bar_sync(1, 32 * max(S, 2));
      // warp 0 finds the bin and its lowest key, warp 1 the highest one; bracketing: warp 0 the first bin's highest
      // key, warp 1 the last one's lowest
      if (warp < 2) {
        const int side = bracketing ? warp : 0, range = r[side];
        int found = -1;
        u64 with = 0, ahead = start;
        if (range >= 0) {
          const u64 base = __shfl_sync(0xffffffffu, inc, range > 0 ? range - 1 : 0);
          const u64 t = of_all(sh.gather[1 + side]), sub = warp_scan(t);
          const int l = __ffs(__ballot_sync(0xffffffffu, reached((range > 0 ? base : 0) + sub, side))) - 1;
          if (!bracketing) {
            with = start + (range > 0 ? base : 0) + __shfl_sync(0xffffffffu, sub, l);
            ahead = with - __shfl_sync(0xffffffffu, t, l);
          }
          found = range * 32 + l;
        }
        const uint32_t under = max(border, K::of(weigh.low) - 1);   // keys from here down: kept by nothing, or no weight
        // lowest key of a bin <= b: the keys about where fp32 has it, else by 32 probes at a time; (none, most], `most` is one
        auto lowest = [&](int b) -> uint32_t {
          uint32_t none = under, most = top_key;
          bool near = true;
          while (most - none > 1) {
            const uint32_t step = (most - none + 31) / 32;
            u64 probe64 = static_cast<u64>(none) + static_cast<u64>(step) * (lane + 1);
            if (near) {
              const uint32_t g = K::of(weigh.top - 2.f * static_cast<float>(b + 1) / (weigh.steps * weigh.more));
              probe64 = static_cast<u64>(max(g, none + 16)) - 15 + lane;
              near = false;
            }
            const uint32_t probe = probe64 < most ? static_cast<uint32_t>(probe64) : most;
            const uint32_t is = __ballot_sync(0xffffffffu, weigh.bin(K::value(probe)) <= b);
            const int first = is ? __ffs(is) - 1 : 32;
            const uint32_t lower = __shfl_sync(0xffffffffu, probe, first > 0 ? first - 1 : 0);
            if (first < 32) most = __shfl_sync(0xffffffffu, probe, first & 31);
            if (first > 0) none = lower;
          }
          return most;
        };
        if (by_key) {
          if (warp == 0 && lane == 0) {
            const uint32_t khi = hi - (static_cast<uint32_t>(found) << shift);
            sh.key_hi = khi;
            sh.key_lo = khi - lo < (1u << shift) ? lo : khi - ((1u << shift) - 1);
          }
        } else if (warp == (bracketing ? 0 : 1)) {
          const uint32_t khi = found > 0 ? lowest(found - 1) - 1 : top_key;
          if (lane == 0) sh.key_hi = khi;
        } else {
          const uint32_t klo = found >= 0 ? lowest(found) : under + 1;   // (bracketing: not surely reached)
          if (lane == 0) sh.key_lo = klo;
        }
        if (warp == 0 && lane == 0) {
          bool missed = bracketing && found < 0;   // not there after all
          if (level == 0 && kind == kBracketed) missed = static_cast<double>(start) >= reach || (found < 0 && lo > under + 1);
          sh.found_at = missed ? -2 : found;
          sh.found_before = ahead;
          sh.found_with = with;
          sh.found_total = total;
          sh.found_count = count;
        }
      }
    }
    __syncthreads();
    buf ^= 1;
    if (bracketing || sh.found_at == -2) {
      if (sh.found_at == -2) above_x = INFINITY;
      kind = sh.found_at == -2 ? kMass : kBracketed;
      lo = sh.key_lo;
      hi = sh.key_hi;
      continue;
    }
    const bool found = sh.found_at >= 0;
    if (mass && level == 0) {
      limit *= static_cast<double>(sh.found_total);
      if (!found) above_x = INFINITY;
    }
    before = found ? sh.found_before : sh.found_total - rest;
    lo = sh.key_lo;
    hi = sh.key_hi;
    if (found && level == 0 && (kind == kMaxima || kind == kMass || (kind == kCount ? sh.found_with : sh.found_count) <= kList)) {
      // the tokens down to the bin's last key into the lists
      const float from_lo = K::value(lo);
      for (int q = q0 + lane; q < q1 && *static_cast<volatile int*>(&sh.listed) <= kList; q += 32) {
        float x[4];
        slice.get(q, x);
        if (!(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= from_lo)) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x[e] >= from_lo) {
            const int at = atomicAdd(&sh.listed, 1);
            if (at < kList)
              sh.list[at] = (static_cast<u64>(K::of(x[e])) << 32) |
                            (0xffffffffu - static_cast<uint32_t>(slice.first + static_cast<long long>(q) * 4 + e));
          }
      }
      row_sync();
      const int count = __reduce_add_sync(0xffffffffu, lane < S ? static_cast<int>(peer32(&sh.listed, lane)) : 0);
      if (count <= kList) {   // (the same in every CTA)
        if (rank == 0) {
          // every thread an entry of one of the lists
          const int c = lane < S ? static_cast<int>(peer32(&sh.listed, lane)) : 0;
          const int end = warp_scan(c);
          int q = 0, first = 0;
          for (int i = 0; i < S - 1; ++i) {
            const int e = __shfl_sync(0xffffffffu, end, i);
            if (tid >= e) {
              q = i + 1;
              first = e;
            }
          }
          if (tid < count) sh.all[tid] = peer64(&sh.list[tid - first], q);
          __syncthreads();
        }
        if (S > 1) cluster_arrive();   // the lists are read
        if (rank == 0) {
          // 1 to 16 lanes an entry, each against its share of the others
          int lanes = 16;
          while (lanes * count > kThreads) lanes >>= 1;
          const int at = tid / lanes, sub = tid % lanes;
          const bool in = at < count;
          const u64 mine = in ? sh.all[at] : 0;
          const float x = K::value(static_cast<uint32_t>(mine >> 32));
          const u64 w = in ? fixed_weight(sh.weigh, x) : 0;
          if (in && sub == 0) sh.weight[at] = w;
          __syncthreads();
          int rank_of = 0;
          u64 over = 0;
          if (in)
#pragma unroll 4
            for (int j = sub; j < count; j += lanes) {
              const bool ahead = sh.all[j] > mine;
              const u64 o = sh.weight[j];
              rank_of += ahead;
              over += ahead ? o : 0;
            }
          for (int off = 1; off < lanes; off <<= 1) {
            rank_of += __shfl_xor_sync(0xffffffffu, rank_of, off);
            over += __shfl_xor_sync(0xffffffffu, over, off);
          }
          bool keep = in && (mass || rank_of < k);
          u64 total;
          if (!mass) {
            block_scan(keep && sub == 0 ? w : 0, sh.red_m, total);
            limit = (by_p ? static_cast<double>(p) : 2.0) * static_cast<double>(total);
          }
          keep = keep && (rank_of == 0 || static_cast<double>(over) < limit) && w >= least;
          __syncthreads();   // the weights are read
          if (in && sub == 0) sh.weight[at] = keep ? w : 0;
          block_scan(keep && sub == 0 ? w : 0, sh.red_m, total);   // (its barriers publish the kept weights)
          const uint32_t code = static_cast<uint32_t>(mine);   // falls as the index rises
          u64 sum = 0;
          if (in)
#pragma unroll 4
            for (int j = sub; j < count; j += lanes) {
              const u64 o = sh.weight[j];
              sum += static_cast<uint32_t>(sh.all[j]) > code ? o : 0;
            }
          for (int off = 1; off < lanes; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          const double target = u * static_cast<double>(total);
          if (keep && sub == 0 && static_cast<double>(sum) <= target && static_cast<double>(sum + w) > target) {
            a.tokens[row] = static_cast<int>(0xffffffffu - code);
            if (a.prob) a.prob[row] = static_cast<float>(real_weight(sh.weigh, x) / static_cast<double>(total));
          }
        }
        if (S > 1) cluster_wait();
        return;
      }
      if (kind == kMaxima) {   // too many: the lists start over
        row_sync();
        if (tid == 0) sh.listed = 0;
        __syncthreads();
      }
    }
    if (kind == kMaxima) {
      kind = kCount;
      before = 0;
      continue;
    }
    ++level;
    if (found && lo != hi) continue;
    if (found) border = lo;
    // (not found: by number, every token with a weight is kept; by mass, the border of top-k stays)
    if (!mass) {
      if (found) ties = k - static_cast<long long>(before);
      if (!by_p) break;
      kind = kBracketing;
      level = 0;
      limit = p;
      before = 0;
      rest_w = border == K::kInf ? 0 : fixed_weight(sh.weigh, K::value(border));
      rest = rest_w ? rest_w * static_cast<u64>(ties) : 0;
      continue;
    }
    // a tie is kept while the mass before it is under the limit
    if (found) {
      ties = a.vocab;
      rest_w = fixed_weight(sh.weigh, K::value(border));
    }
    if (rest_w > 0) {
      long long c = static_cast<long long>((limit - static_cast<double>(before)) / static_cast<double>(rest_w));
      c = c < 0 ? 0 : c;
      while (c > 0 && static_cast<double>(before + static_cast<u64>(c - 1) * rest_w) >= limit) --c;
      while (c < a.vocab && static_cast<double>(before + static_cast<u64>(c) * rest_w) < limit) ++c;
      ties = c < ties ? c : ties;
    }
    break;
  }

  // ------------------------------------------------------------------- the token --
  const float border_x = K::value(border);
  const float cut = over_border();
  const bool filtered = border != K::kInf || least > 0 || !weigh.plain();
  u64 border_w = 0;
  if (border != K::kInf && border_x >= weigh.low) border_w = fixed_weight(sh.weigh, border_x);
  // the mass over the bracket is known already, if min-p takes nothing of it
  const bool known = above_x != INFINITY && border_w >= least;
  if (border_w < least) border_w = 0;
  // mass over the border and ties of each warp's part of the slice
  {
    u64 s = 0;
    int c = 0;
    if (!filtered) {
      int quads = 0;
      for (int q = q0 + lane; q < q1; q += 32, ++quads) {
        float x[4];
        slice.get(q, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) s += weigh.biased(x[e]);
      }
      s -= static_cast<u64>(quads * 4) * Weigh::kBias;
    } else {
      for (int q = q0 + lane; q < q1; q += 32) {
        float x[4];
        slice.get(q, x);
        for (int e = 0; e < 4; ++e) c += x[e] == border_x;
        bool in[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) in[e] = x[e] >= cut && (!known || x[e] <= above_x);
        if (!(in[0] || in[1] || in[2] || in[3])) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u64 w = weigh.biased(x[e], in[e]) - Weigh::kBias;
          s += w >= least ? w : 0;
        }
      }
    }
    if (known) s += above;
    s = warp_sum(s);
    c = warp_sum(c);
    if (lane == 0) {
      sh.part_mass[warp] = s;
      sh.part_ties[warp] = c;
    }
  }
  row_sync();
  if (warp == 0) {   // the part with the token: a lane has up to 4 of the parts in a row
    const int per = max(1, S * kWarps / 32);
    u64 m[4];
    int t[4], t_sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // (every fetch of another CTA's before the first use)
      const int part = min(lane * per + j, S * kWarps - 1);
      const u64* const pm = &sh.part_mass[part % kWarps];
      const int* const pt = &sh.part_ties[part % kWarps];
      m[j] = S == 1 ? *pm : 0;
      t[j] = S == 1 ? *pt : 0;
      if (S > 1) {
        m[j] = ld_dsmem_u64(dsmem_addr(smem_u32(pm), part / kWarps));
        t[j] = static_cast<int>(ld_dsmem_u32(dsmem_addr(smem_u32(pt), part / kWarps)));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= per || lane * per + j >= S * kWarps) {
        m[j] = 0;
        t[j] = 0;
      }
      t_sum += t[j];
    }
    int t_before = warp_scan(t_sum) - t_sum;
    u64 sum = 0;
    int tb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      tb[j] = t_before;
      const long long left = ties - t_before;
      m[j] += static_cast<u64>(left < 0 ? 0 : left < t[j] ? left : t[j]) * border_w;
      sum += m[j];
      t_before += t[j];
    }
    const u64 inc = warp_scan(sum);
    const u64 total = __shfl_sync(0xffffffffu, inc, 31);
    const double target = u * static_cast<double>(total);
    const int at = __ffs(__ballot_sync(0xffffffffu, static_cast<double>(inc) > target)) - 1;
    if (lane == at) {
      u64 ahead = inc - sum;
      int j = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (j == i && static_cast<double>(ahead + m[i]) <= target) {
          ahead += m[i];
          ++j;
        }
      sh.at_part = lane * per + j;
      sh.at_before = ahead;
      sh.at_ties = j == 0 ? tb[0] : j == 1 ? tb[1] : j == 2 ? tb[2] : tb[3];
      sh.total = total;
      sh.target = target;
      sh.done = 0;
    }
  }
  __syncthreads();
  if (S > 1) cluster_arrive();   // this CTA has read what it needs of its peers
  if (sh.at_part / kWarps == rank) {
    // the token's part once more, a quad per thread
    const int qa = sh.at_part % kWarps * (a.part * (n / 4)), qb = qa + a.part * (n / 4);
    u64 ahead = sh.at_before;
    long long ties_ahead = sh.at_ties;
    const double target = sh.target;
    for (int qi = qa; qi < qb; qi += kThreads) {
      const int q = qi + tid;
      float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      u64 w[4];
      int c = 0;
      if (q < qb) slice.get(q, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) c += q < qb && x[e] == border_x;
      int n_ties = 0, tie = 0;
      if (filtered) tie = block_scan(c, sh.red_c, n_ties);
      u64 s = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = 0;
        if (x[e] >= cut) {
          w[e] = fixed_weight(sh.weigh, x[e]);
          w[e] = w[e] >= least ? w[e] : 0;
        }
        if (filtered && q < qb && x[e] == border_x && ties_ahead + tie++ < ties) w[e] = border_w;
        s += w[e];
      }
      u64 part_mass;
      u64 sum = ahead + block_scan(s, sh.red_m, part_mass);
      if (static_cast<double>(sum) <= target && static_cast<double>(sum + s) > target) {   // one thread's
        int e = 0;
        while (static_cast<double>(sum + w[0]) <= target) {   // (its sum exceeds the target: e stays under 4)
          sum += w[0];
          w[0] = w[1];
          w[1] = w[2];
          w[2] = w[3];
          x[0] = x[1];
          x[1] = x[2];
          x[2] = x[3];
          ++e;
        }
        a.tokens[row] = static_cast<int>(slice.first + static_cast<long long>(q) * 4 + e);
        if (a.prob) a.prob[row] = static_cast<float>(real_weight(sh.weigh, x[0]) / static_cast<double>(sh.total));
        sh.done = 1;
      }
      __syncthreads();
      if (sh.done) break;
      ahead += part_mass;
      ties_ahead += n_ties;
    }
  }
  if (S > 1) cluster_wait();
}

template <typename T>
cudaError_t launch(cudaStream_t st, SampleArgs a, int sms) {
  constexpr int n = Key<T>::n;
  constexpr size_t kMost = 200 * 1024;
  const long long vectors = (static_cast<long long>(a.vocab) + 2 * (n - 1)) / n;   // with a row's skew
  a.head = static_cast<int>(a.top_k || a.top_p ? kHeadFull : kHeadPlain);
  // CTAs per row: so that two of them, slices and all, fit an SM's shared memory; more while the machine
  // has room for them and each keeps 4096 logits.  Many rows without a border to find: 8-warp CTAs of up to 52 KB, four
  // an SM, so that one loads while others weigh (300 bf16 rows of 151936: 86 -> 80 us).
  int S = 1, warps = 16;
  while (S < kMaxS && vectors * 16 > S * 80 * 1024LL) S *= 2;
  while (S < kMaxS && 2LL * S * a.rows <= 2LL * sms && a.vocab >= 2 * S * 4096) S *= 2;
  if (!a.top_k && !a.top_p && vectors * 16 <= kMaxS * 52 * 1024LL && 1LL * S * a.rows > 2LL * sms) {
    warps = 8;
    while (S < kMaxS && vectors * 16 > S * 52 * 1024LL) S *= 2;
  }
  a.S = S;
  a.part = static_cast<int>((vectors + S * warps - 1) / (S * warps));
  const size_t bytes = a.head + static_cast<size_t>(a.part) * warps * 16;
  const bool staged = bytes <= kMost;
  if (!staged) {   // (slices of 2^16 logits at most, as the histogram's counters need)
    warps = 16;
    a.part = static_cast<int>((vectors + S * warps - 1) / (S * warps));
  }
  auto* kernel = !staged ? sample_kernel<T, false, 16> : warps == 16 ? sample_kernel<T, true, 16> : sample_kernel<T, true, 8>;
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  static std::atomic<bool> ready[64];   // per device: the staged kernels' shared-memory limit
  if (staged && (dev >= 64 || !ready[dev].load(std::memory_order_acquire))) {
    for (auto* k : {sample_kernel<T, true, 16>, sample_kernel<T, true, 8>})
      if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost)) != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * S);
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = staged ? bytes : a.head;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_sample(cudaStream_t st, const SampleArgs& a, int dtype, int sms) {
  return dtype == NLD_F32 ? launch<float>(st, a, sms) : launch<__nv_bfloat16>(st, a, sms);
}

}  // namespace nld
