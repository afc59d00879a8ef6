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
// in the order of falling logits: the first over equal steps of (max x - x) / T, kPerOctave per
// halving of the weight; the next over the order-preserving keys inside the border's bin, until
// that bin is one key (three levels for fp32, two for bf16, whatever the values).  Every
// CTA counts its slice; one cluster barrier later each of them finds the bin from all CTAs'
// range sums and that range's bins over distributed shared memory.
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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxS = 8;            // CTAs of a row
constexpr int kBins = 1024;
constexpr int kRanges = 32;         // of 32 bins
constexpr float kPerOctave = 20.f;  // bins per halving: the last one starts at 2^-51, no weight
constexpr double kOne = 17592186044416.0;   // 2^44: the weight of the largest logit

typedef unsigned long long u64;

// Keys in the order of the values, of as many bits as the type has; -inf has the key kInf.
template <typename T>
struct Key;
template <>
struct Key<float> {
  static constexpr int n = 4;   // logits per 16 bytes
  static constexpr uint32_t kInf = 0x007fffffu;
  static NLD_DEV uint32_t of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  }
  static NLD_DEV float value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }
  static NLD_DEV void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static NLD_DEV uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Key<__nv_bfloat16> {
  static constexpr int n = 8;
  static constexpr uint32_t kInf = 0x007fu;
  static NLD_DEV uint32_t of(float x) { return Key<float>::of(x) >> 16; }
  static NLD_DEV float value(uint32_t k) {
    return __uint_as_float((k & 0x8000u) ? (k ^ 0x8000u) << 16 : (k ^ 0xffffu) << 16);
  }
  static NLD_DEV void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static NLD_DEV uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (__float_as_uint(x[2 * i]) >> 16) | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
// NaN counts as -inf, -0 as +0 (equal values must have equal keys).
NLD_DEV float plain_logit(float v) { return (v == v) ? v + 0.f : -INFINITY; }

// Weights of a row's logits.
struct Weigh {
  float top, half_top;
  float steps, more;  // their product: bins of the first level per unit of (max x - x) / 2
  double top_d, inv_t, s16;
  const double* tab;  // 2^(j / 16), j = 0..15
  NLD_DEV void init(float top_, float temperature, const double* tab_) {
    top = top_;
    half_top = 0.5f * top_;   // halves: the difference of two finite logits may exceed fp32
    top_d = static_cast<double>(top_);
    inv_t = 1.0 / static_cast<double>(temperature);
    s16 = inv_t * 23.083120654223414;   // 16 log2(e)
    const double per = inv_t * (2.0 * 1.4426950408889634 * kPerOctave);
    steps = static_cast<float>(fmin(per, 1e38));
    more = per > 1e38 ? static_cast<float>(per / 1e38) : 1.f;
    tab = tab_;
  }
  // Bin of the first level: whole, not falling as x falls; kBins - 1: no weight (-inf, and all but the
  // largest where that is +inf).
  NLD_DEV int bin(float x) const {
    if (x == top) return 0;
    const float d = (half_top - 0.5f * x) * steps * more;
    return d < static_cast<float>(kBins - 1) ? static_cast<int>(d) : kBins - 1;   // (inf, and 0 x inf = NaN: the last)
  }
  NLD_DEV double real(float x) const {
    if (x == top) return 1.0;
    if (bin(x) == kBins - 1) return 0.0;
    return exp((static_cast<double>(x) - top_d) * inv_t);
  }
  // exp((x - top) / T) 2^44, rounded, of an x that is not in the last bin.  With y = 16 log2(e) (x - top) / T
  // = k + r, |r| <= 1/2: 2^(y / 16) = 2^(k / 16) p(r), p the Chebyshev interpolant of degree 5 of 2^(r / 16)
  // with p(0) set to 1: within 2^-46 of it.  y is rounded, and w converted, by adding 2^52 and more.
  NLD_DEV u64 fixed(float x) const {
    constexpr double kRound = 6755399441055744.0;   // 1.5 2^52: whole numbers in the low word
    const double d = x == top ? 0.0 : static_cast<double>(x) - top_d;
    const double t = fma(d, s16, kRound);
    const double r = fma(d, s16, kRound - t);
    const int k = __double2loint(t);
    double p = fma(r, 1.2716085030349987e-09, 1.4676444621898709e-07);
    p = fma(r, p, 1.355080777749983e-05);
    p = fma(r, p, 0.000938384792486206);
    p = fma(r, p, 0.043321698784996608);
    p = fma(r, p, 1.0);
    const double m = tab[k & 15];
    const double scaled = __hiloint2double(__double2hiint(m) + (((k >> 4) + 44) << 20), __double2loint(m));
    return static_cast<u64>(__double_as_longlong(fma(scaled, p, 4503599627370496.0))) & 0x000fffffffffffffull;
  }
};

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
// Sum over the threads before this one, and over all.  `red` holds kWarps entries; callable again at
// once.
template <typename V>
NLD_DEV V block_scan(V v, V* red, V& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const V inc = warp_scan(v);
  __syncthreads();
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  const V w = lane < kWarps ? red[lane] : V(0);
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
template <bool kValue>
struct Flag {
  static constexpr bool value = kValue;
};

// What a CTA's peers read, and its own scratch.
struct Shared {
  uint32_t hist[2][3][kBins];   // [buffer][limb][bin]; counts use limb 0
  u64 range[2][kRanges];        // [buffer]: sums over 32 bins
  u64 best;                     // the slice's largest key and the complement of its lowest index
  u64 part_mass[kWarps];        // kept mass over the border, ties at it: of each warp's part of the slice
  int part_ties[kWarps];
  double tab[16];
  u64 red_m[kWarps];
  int red_c[kWarps];
  u64 found_before;             // warp 0's findings
  u64 found_total;
  int found_at;
  uint32_t key_lo, key_hi;
  int at_part, done;            // the sampled token's part, and what lies before that part
  u64 at_before, total;
  long long at_ties;
  double target;
};

// One row's slice: the 16-byte vectors of it, in shared memory or (slices over the shared memory)
// straight from global memory.
template <typename T, bool kStaged>
struct Slice {
  static constexpr int n = Key<T>::n;
  const uint4* staged;
  const T* row;
  long long first;    // index of the slice's first logit (a 16-byte boundary; before the row's start by up to n - 1)
  int vocab;
  NLD_DEV bool whole(int v) const {
    const long long i0 = first + static_cast<long long>(v) * n;
    return i0 >= 0 && i0 + n <= vocab;
  }
  NLD_DEV uint4 raw(int v) const { return __ldg(reinterpret_cast<const uint4*>(row + (first + static_cast<long long>(v) * n))); }
  // plain_logit of the logits of vector v, read as `got` where it is whole; -inf outside the row
  NLD_DEV void plain(int v, const uint4& got, float (&x)[n]) const {
    if (whole(v)) {
      Key<T>::unpack(got, x);
#pragma unroll
      for (int e = 0; e < n; ++e) x[e] = plain_logit(x[e]);
    } else {
      const long long i0 = first + static_cast<long long>(v) * n;
#pragma unroll
      for (int e = 0; e < n; ++e) x[e] = i0 + e >= 0 && i0 + e < vocab ? plain_logit(to_f32<T>(row[i0 + e])) : -INFINITY;
    }
  }
  NLD_DEV void get(int v, float (&x)[n]) const {
    if constexpr (kStaged) Key<T>::unpack(staged[v], x);
    else plain(v, whole(v) ? raw(v) : make_uint4(0, 0, 0, 0), x);
  }
};

template <typename T, bool kStaged>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  using K = Key<T>;
  constexpr int n = K::n;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  constexpr size_t kHead = (sizeof(Shared) + 15) / 16 * 16;
  const int S = a.S, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % S;
  const size_t row = blockIdx.x / S;
  Slice<T, kStaged> slice;
  slice.staged = reinterpret_cast<const uint4*>(smem + kHead);
  slice.row = static_cast<const T*>(a.logits) + row * a.ld;
  slice.vocab = a.vocab;
  // the row's vectors start at the 16-byte boundary at or before it; warp w of the slice has a.part of them
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(slice.row) % 16 / sizeof(T));
  slice.first = static_cast<long long>(rank) * (a.part * kWarps * n) - skew;
  const int v0 = warp * a.part, v1 = v0 + a.part;
  const uint32_t sh_base = smem_u32(&sh);

  for (int i = tid; i < 2 * 3 * kBins; i += kThreads) (&sh.hist[0][0][0])[i] = 0;
  if (tid < 16) sh.tab[tid] = exp2(tid * 0.0625);

  // the largest logit, and the lowest index that has it
  {
    float big = -INFINITY;
    int at = 0x7fffffff;
    constexpr int kU = 8;   // vectors in flight
    for (int vb = v0 + lane; vb < v1; vb += 32 * kU) {
      uint4 got[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (vb + 32 * u < v1 && slice.whole(vb + 32 * u)) got[u] = slice.raw(vb + 32 * u);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int v = vb + 32 * u;
        if (v >= v1) break;
        float x[n];
        slice.plain(v, got[u], x);
        if constexpr (kStaged) reinterpret_cast<uint4*>(smem + kHead)[v] = K::pack(x);
#pragma unroll
        for (int e = 0; e < n; ++e)
          if (x[e] > big) {
            big = x[e];
            at = v * n + e;
          }
      }
    }
    u64 best = (static_cast<u64>(K::of(big)) << 32) |
               (big == -INFINITY ? 0u : 0xffffffffu - static_cast<uint32_t>(slice.first + at));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const u64 o = __shfl_xor_sync(0xffffffffu, best, off);
      best = o > best ? o : best;
    }
    if (lane == 0) sh.red_m[warp] = best;
    __syncthreads();
    if (warp == 0) {
      best = lane < kWarps ? sh.red_m[lane] : 0;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const u64 o = __shfl_xor_sync(0xffffffffu, best, off);
        best = o > best ? o : best;
      }
      if (lane == 0) sh.best = best;
    }
  }
  cluster_sync();
  u64 best = lane < S ? ld_dsmem_u64(dsmem_addr(smem_u32(&sh.best), lane)) : 0;
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) {
    const u64 o = __shfl_xor_sync(0xffffffffu, best, off);
    best = o > best ? o : best;
  }
  best = __shfl_sync(0xffffffffu, best, 0);
  const uint32_t top_key = static_cast<uint32_t>(best >> 32);
  const float temperature = a.temperature ? a.temperature[row] : 1.f;
  if (top_key == K::kInf || !(temperature > 0.f)) {   // (the same for the whole cluster)
    if (rank == 0 && tid == 0) {
      a.tokens[row] = top_key == K::kInf ? -1 : static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
      if (a.prob) a.prob[row] = top_key == K::kInf ? 0.f : 1.f;
    }
    cluster_sync();   // peers may still be reading sh.best
    return;
  }
  Weigh weigh;
  weigh.init(K::value(top_key), temperature, sh.tab);

  // Border among the tokens with keys over kept_over: the key with which their number (by mass: their mass)
  // in falling order reaches `limit` (by mass: that share of `total`, which is their mass and `rest`).  False
  // if none of those with a weight does; else `key`, and in `before` what lies over it.
  int buf = 0;
  auto find = [&](auto by_mass, uint32_t kept_over, u64 rest, double limit, uint32_t& key, u64& before, u64& total) -> bool {
    constexpr bool kMass = decltype(by_mass)::value;
    uint32_t lo = 0, hi = 0;   // keys of the current bin
    before = 0;
    for (int level = 0;; ++level) {
      uint32_t(*h)[kBins] = sh.hist[buf];
      int shift = 0;
      if (level > 0)
        while (((hi - lo) >> shift) >= kBins) ++shift;
      for (int v = v0 + lane; v < v1; v += 32) {
        float x[n];
        slice.get(v, x);
#pragma unroll
        for (int e = 0; e < n; ++e) {
          int b;
          bool in;
          if (level == 0) {
            b = weigh.bin(x[e]);
            in = b < kBins - 1 && (!kMass || K::of(x[e]) > kept_over);
          } else {
            const uint32_t k = K::of(x[e]);
            in = k >= lo && k <= hi;
            b = static_cast<int>((hi - k) >> shift);
          }
          if (!in) continue;
          if constexpr (kMass) {
            const u64 w = weigh.fixed(x[e]);
            const uint32_t w2 = static_cast<uint32_t>(w >> 30), w1 = static_cast<uint32_t>(w >> 15) & 0x7fffu;
            atomicAdd(&h[0][b], static_cast<uint32_t>(w) & 0x7fffu);
            if (w1) atomicAdd(&h[1][b], w1);
            if (w2) atomicAdd(&h[2][b], w2);
          } else {
            atomicAdd(&h[0][b], 1u);
          }
        }
      }
      __syncthreads();
      auto bin_sum = [&](uint32_t base, int b) -> u64 {   // of one CTA, at its shared-window address
        const uint32_t p = base + static_cast<uint32_t>(reinterpret_cast<uint8_t*>(&h[0][0]) - smem) + b * 4;
        u64 s = ld_dsmem_u32(p);
        if constexpr (kMass)
          s += (static_cast<u64>(ld_dsmem_u32(p + kBins * 4)) << 15) + (static_cast<u64>(ld_dsmem_u32(p + 2 * kBins * 4)) << 30);
        return s;
      };
      const uint32_t own = dsmem_addr(sh_base, rank);
      for (int r = warp; r < kRanges; r += kWarps) {
        const u64 s = warp_sum(bin_sum(own, r * 32 + lane));
        if (lane == 0) sh.range[buf][r] = s;
      }
      cluster_sync();
      // the other buffer was last read before this barrier
      for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[buf ^ 1][0][0])[i] = 0;
      if (warp == 0) {
        u64 s = 0;
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uint8_t*>(&sh.range[buf][lane]) - smem);
#pragma unroll
        for (int q = 0; q < kMaxS; ++q)
          if (q < S) s += ld_dsmem_u64(dsmem_addr(sh_base, q) + at);
        u64 inc = warp_scan(s);
        if (level == 0) {
          total = __shfl_sync(0xffffffffu, inc, 31) + rest;
          if (kMass) limit *= static_cast<double>(total);   // (warp 0 alone compares with it)
        }
        auto reached = [&](u64 c) { return static_cast<double>(before + c) >= limit; };
        uint32_t m = __ballot_sync(0xffffffffu, reached(inc));
        int found = -1;
        if (m) {
          const int r = __ffs(m) - 1;
          const u64 base = __shfl_sync(0xffffffffu, inc - s, r);
          u64 t = 0;
#pragma unroll
          for (int q = 0; q < kMaxS; ++q)
            if (q < S) t += bin_sum(dsmem_addr(sh_base, q), r * 32 + lane);
          inc = warp_scan(t);
          m = __ballot_sync(0xffffffffu, reached(base + inc));
          const int l = __ffs(m) - 1;
          before += base + __shfl_sync(0xffffffffu, inc - t, l);
          found = r * 32 + l;
        }
        // the keys of that bin
        uint32_t klo = 0, khi = 0;
        if (found >= 0 && level == 0) {
          // lowest key of a bin <= b, by 32 probes at a time: keys (from, to], `to` is one
          auto lowest = [&](int b) -> uint32_t {
            uint32_t from = K::kInf, to = top_key;
            while (to - from > 1) {
              const uint32_t step = (to - from + 31) / 32;
              const u64 probe64 = static_cast<u64>(from) + static_cast<u64>(step) * (lane + 1);
              const uint32_t probe = probe64 < to ? static_cast<uint32_t>(probe64) : to;
              const int first = __ffs(__ballot_sync(0xffffffffu, weigh.bin(K::value(probe)) <= b)) - 1;
              const uint32_t got = __shfl_sync(0xffffffffu, probe, first);
              from = first > 0 ? __shfl_sync(0xffffffffu, probe, first - 1) : from;
              to = got;
            }
            return to;
          };
          klo = lowest(found);
          klo = klo > kept_over ? klo : kept_over + 1;
          khi = found > 0 ? lowest(found - 1) - 1 : top_key;
        } else if (found >= 0) {
          khi = hi - (static_cast<uint32_t>(found) << shift);
          klo = khi - lo < (1u << shift) ? lo : khi - ((1u << shift) - 1);
        }
        if (lane == 0) {
          sh.found_at = found;
          sh.found_before = before;
          sh.found_total = total;
          sh.key_lo = klo;
          sh.key_hi = khi;
        }
      }
      __syncthreads();
      buf ^= 1;
      before = sh.found_before;
      total = sh.found_total;
      lo = sh.key_lo;
      hi = sh.key_hi;
      if (sh.found_at < 0) return false;
      if (lo == hi) {
        key = lo;
        return true;
      }
    }
  };

  // kept: keys over `border`, and the first `ties` tokens at it
  uint32_t border = K::kInf;
  long long ties = a.vocab;
  u64 over = 0, total = 0;
  const int k = a.top_k ? a.top_k[row] : 0;
  if (k > 0 && k < a.vocab && find(Flag<false>(), K::kInf, 0, k, border, over, total)) ties = k - static_cast<long long>(over);
  const float p = a.top_p ? a.top_p[row] : 1.f;
  if (p <= 0.f) {   // p of nothing: the likeliest token alone
    border = top_key;
    ties = 1;
  } else if (p < 1.f) {
    const u64 at_border = border == K::kInf ? 0 : weigh.fixed(K::value(border)) * static_cast<u64>(ties);
    uint32_t key = border;
    const bool below = find(Flag<true>(), border, at_border, p, key, over, total);
    const double limit = static_cast<double>(p) * static_cast<double>(total);
    if (below) ties = a.vocab;
    else over = total - at_border;
    border = key;
    // a tie is kept while the mass before it is under the limit
    const u64 w = border == K::kInf ? 0 : weigh.fixed(K::value(border));
    if (w > 0) {
      long long c = static_cast<long long>((limit - static_cast<double>(over)) / static_cast<double>(w));
      c = c < 0 ? 0 : c;
      while (c > 0 && static_cast<double>(over + static_cast<u64>(c - 1) * w) >= limit) --c;
      while (c < a.vocab && static_cast<double>(over + static_cast<u64>(c) * w) < limit) ++c;
      ties = c < ties ? c : ties;
    }
  }
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  const double least = mp > 0.f ? static_cast<double>(fminf(mp, 1.f)) * kOne : 0.0;
  auto kept_mass = [&](float x) -> u64 {   // of a token over the border
    if (weigh.bin(x) == kBins - 1) return 0;
    const u64 w = weigh.fixed(x);
    return static_cast<double>(w) >= least ? w : 0;
  };
  const u64 border_w = border == K::kInf ? 0 : kept_mass(K::value(border));

  // mass over the border and ties of each warp's part of the slice
  {
    u64 s = 0;
    int c = 0;
    for (int v = v0 + lane; v < v1; v += 32) {
      float x[n];
      slice.get(v, x);
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const uint32_t key = K::of(x[e]);
        if (key > border) s += kept_mass(x[e]);
        c += key == border;
      }
    }
    s = warp_sum(s);
    c = warp_sum(c);
    if (lane == 0) {
      sh.part_mass[warp] = s;
      sh.part_ties[warp] = c;
    }
  }
  cluster_sync();
  if (warp == 0) {   // the part with the token: a lane has up to 4 of the parts in a row
    const int per = S >= 2 ? S / 2 : 1;
    u64 m[4];
    int t[4], t_sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int part = lane * per + j;
      m[j] = 0;
      t[j] = 0;
      if (j < per && part < S * kWarps) {
        const uint32_t peer = dsmem_addr(sh_base, part / kWarps);
        m[j] = ld_dsmem_u64(peer + static_cast<uint32_t>(offsetof(Shared, part_mass)) + (part % kWarps) * 8);
        t[j] = static_cast<int>(ld_dsmem_u32(peer + static_cast<uint32_t>(offsetof(Shared, part_ties)) + (part % kWarps) * 4));
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
    total = __shfl_sync(0xffffffffu, inc, 31);
    const float uf = a.u[row];
    const double target = (uf > 0.f ? static_cast<double>(fminf(uf, 0.99999994f)) : 0.0) * static_cast<double>(total);
    const int at = __ffs(__ballot_sync(0xffffffffu, static_cast<double>(inc) > target)) - 1;
    if (lane == at) {
      u64 before = inc - sum;
      int j = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (j == i && static_cast<double>(before + m[i]) <= target) {
          before += m[i];
          ++j;
        }
      sh.at_part = lane * per + j;
      sh.at_before = before;
      sh.at_ties = j == 0 ? tb[0] : j == 1 ? tb[1] : j == 2 ? tb[2] : tb[3];
      sh.total = total;
      sh.target = target;
      sh.done = 0;
    }
  }
  __syncthreads();
  cluster_arrive();   // this CTA has read what it needs of its peers
  const int at_part = sh.at_part % kWarps;
  if (sh.at_part / kWarps == rank) {
    // the token's part once more, a vector per thread
    u64 before = sh.at_before;
    long long ties_before = sh.at_ties;
    const double target = sh.target;
    for (int i0 = 0; i0 < a.part; i0 += kThreads) {
      const bool in = i0 + tid < a.part;
      const int v = at_part * a.part + i0 + tid;
      float x[n];
      u64 w[n];
      int c = 0;
      if (in) slice.get(v, x);
#pragma unroll
      for (int e = 0; e < n; ++e) c += in && K::of(x[e]) == border;
      int n_ties;
      int tie = block_scan(c, sh.red_c, n_ties);
      u64 s = 0;
#pragma unroll
      for (int e = 0; e < n; ++e) {
        w[e] = 0;
        if (in) {
          const uint32_t key = K::of(x[e]);
          if (key > border) w[e] = kept_mass(x[e]);
          if (key == border && ties_before + tie++ < ties) w[e] = border_w;
        }
        s += w[e];
      }
      u64 mass;
      u64 sum = before + block_scan(s, sh.red_m, mass);
      if (static_cast<double>(sum) <= target && static_cast<double>(sum + s) > target) {   // one thread's
        bool open = true;
#pragma unroll
        for (int e = 0; e < n; ++e) {
          sum += w[e];
          if (open && static_cast<double>(sum) > target) {
            open = false;
            a.tokens[row] = static_cast<int>(slice.first + static_cast<long long>(v) * n + e);
            if (a.prob) a.prob[row] = static_cast<float>(weigh.real(x[e]) * kOne / static_cast<double>(sh.total));
          }
        }
        sh.done = 1;
      }
      __syncthreads();
      if (sh.done) break;
      before += mass;
      ties_before += n_ties;
    }
  }
  cluster_wait();
}

template <typename T>
cudaError_t launch(cudaStream_t st, SampleArgs a, int sms) {
  constexpr int n = Key<T>::n;
  constexpr size_t kHead = (sizeof(Shared) + 15) / 16 * 16;
  const long long vectors = (static_cast<long long>(a.vocab) + 2 * (n - 1)) / n;   // with a row's skew
  // CTAs per row: so that two of them, slices and all, fit an SM's shared memory; more while the machine
  // has room for them and each keeps 4096 logits
  int S = 1;
  while (S < kMaxS && vectors * 16 > S * 80 * 1024LL) S *= 2;
  while (S < kMaxS && 2LL * S * a.rows <= 2LL * sms && a.vocab >= 2 * S * 4096) S *= 2;
  a.S = S;
  a.part = static_cast<int>((vectors + S * kWarps - 1) / (S * kWarps));
  const size_t bytes = kHead + static_cast<size_t>(a.part) * kWarps * 16;
  const bool staged = bytes <= 200 * 1024;
  auto* kernel = staged ? sample_kernel<T, true> : sample_kernel<T, false>;
  cudaError_t e;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  static std::atomic<bool> ready[64];   // per device: the staged kernel's shared-memory limit
  if (staged && (dev >= 64 || !ready[dev].load(std::memory_order_acquire))) {
    if ((e = cudaFuncSetAttribute(sample_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024)) != cudaSuccess)
      return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * S);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = staged ? bytes : kHead;
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
