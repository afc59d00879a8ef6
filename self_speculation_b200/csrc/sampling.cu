// The next token of every row of logits from a given uniform number (nld_sample).
//
// With x the row's logits and T its temperature, w_i = exp((x_i - max x) / T).  In the order of
// falling logits, equal ones by index: top-k keeps the first k tokens; top-p the tokens of these
// before which less than p of their mass lies (one at least); min-p the tokens of these with
// w_i >= min_p.  The sampled token is the first kept one, by index, up to and with which more than
// u of the kept mass lies.
//
// The kept tokens are those whose logit exceeds a border value and the first few, by index, that
// equal it; a border is found by a search over the 32 bits of the logits' order-preserving
// keys.  Masses are sums of 64-bit fixed-point weights (2^44 at the row's largest logit, from exp in
// 64 bits; up to 2^19 tokens fit): their sums do not depend on the order of addition, so neither
// do the borders or the token.
#include "common.cuh"

namespace nld {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr double kOne = 17592186044416.0;   // 2^44: the weight of the largest logit

typedef unsigned long long u64;

// Logit i of a row: NaN counts as -inf, -0 as +0 (equal values must have equal keys).
template <typename T>
NLD_DEV float load_logit(const T* x, int i) {
  const float v = to_f32<T>(x[i]);
  return (v == v) ? v + 0.f : -INFINITY;
}
// Keys in the order of the values; -inf has the key kInfKey.
NLD_DEV uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
NLD_DEV float value_of(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }
constexpr uint32_t kInfKey = 0x007fffffu;

struct Weigh {
  double top, inv_t;
  NLD_DEV double real(uint32_t key) const {
    const float x = value_of(key);
    if (x == static_cast<float>(top)) return 1.0;
    if (x == -INFINITY || top == INFINITY) return 0.0;
    return exp((static_cast<double>(x) - top) * inv_t);
  }
  NLD_DEV u64 operator()(uint32_t key) const { return __double2ull_rn(real(key) * kOne); }
};

template <typename V>
NLD_DEV V warp_sum(V v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// Sum over the block, to every thread.  `red` holds kWarps entries; callable again at once.
template <typename V>
NLD_DEV V block_sum(V v, V* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(red[threadIdx.x & 31]);
}
// Sum over the threads before this one.
template <typename V>
NLD_DEV V block_scan(V v, V* red, V& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const V o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  __syncthreads();
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  const V w = red[lane];
  V before = warp_sum(lane < warp ? w : V(0));
  total = warp_sum(w);
  return before + inc - v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  static_assert(kWarps == 32, "one warp reduces the warps' values");
  __shared__ u64 red_m[kWarps];
  __shared__ int red_c[kWarps];
  __shared__ u64 seg_mass[kWarps];
  __shared__ int seg_ties[kWarps];
  __shared__ int s_token;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* x = static_cast<const T*>(a.logits) + static_cast<size_t>(row) * a.ld;
  const int V = a.vocab;

  // the largest logit, and the lowest index that has it
  u64 best = 0;   // key, then the index's complement
  for (int i = tid; i < V; i += kThreads) {
    const u64 c = (static_cast<u64>(key_of(load_logit(x, i))) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
    best = c > best ? c : best;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const u64 o = __shfl_xor_sync(0xffffffffu, best, off);
    best = o > best ? o : best;
  }
  if (lane == 0) red_m[warp] = best;
  __syncthreads();
  best = red_m[lane];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const u64 o = __shfl_xor_sync(0xffffffffu, best, off);
    best = o > best ? o : best;
  }
  const uint32_t top_key = static_cast<uint32_t>(best >> 32);
  const int top_at = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
  const float temperature = a.temperature ? a.temperature[row] : 1.f;
  if (top_key == kInfKey || !(temperature > 0.f)) {
    if (tid == 0) {
      a.tokens[row] = top_key == kInfKey ? -1 : top_at;
      if (a.prob) a.prob[row] = top_key == kInfKey ? 0.f : 1.f;
    }
    return;
  }
  Weigh weigh;
  weigh.top = static_cast<double>(value_of(top_key));
  weigh.inv_t = 1.0 / static_cast<double>(temperature);

  auto count_from = [&](uint32_t key) {   // tokens whose key is `key` or more
    int c = 0;
    for (int i = tid; i < V; i += kThreads) c += key_of(load_logit(x, i)) >= key;
    return block_sum(c, red_c);
  };
  auto mass_over = [&](uint32_t key) {   // mass of the tokens whose key is over `key`
    u64 s = 0;
    for (int i = tid; i < V; i += kThreads) {
      const uint32_t k = key_of(load_logit(x, i));
      if (k > key) s += weigh(k);
    }
    return block_sum(s, red_m);
  };

  // kept: keys over `border`, and the first `ties` tokens at it
  uint32_t border = kInfKey;
  long long ties = V;
  const int k = a.top_k ? a.top_k[row] : 0;
  if (k > 0 && k < V) {
    // the largest key that at least k tokens reach
    uint32_t b = 0;
    for (int bit = 31; bit >= 0; --bit)
      if (count_from(b | (1u << bit)) >= k) b |= 1u << bit;
    if (b > kInfKey) {
      border = b;
      ties = k - (b == 0xffffffffu ? 0 : count_from(b + 1));
    }
  }
  const float p = a.top_p ? a.top_p[row] : 1.f;
  if (p < 1.f) {
    const int at_border = count_from(border) - count_from(border + 1);
    const u64 total = mass_over(border) + weigh(border) * static_cast<u64>(ties < at_border ? ties : at_border);
    const double limit = static_cast<double>(p) * static_cast<double>(total);
    if (!(limit > 0.0)) {   // p of nothing: the likeliest token alone
      border = top_key;
      ties = 1;
    } else {
      // the smallest key from the border on that less than the limit lies over
      uint32_t b = 0;   // the largest key below which the limit is reached, plus one
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = (b | (1u << bit)) - 1;
        if (c < border || static_cast<double>(mass_over(c)) >= limit) b |= 1u << bit;
      }
      if (b > border) {
        border = b;
        ties = V;
      }
      // a tie is kept while the mass before it is under the limit
      const u64 over = mass_over(border), w = weigh(border);
      long long n = V;
      if (w > 0) {
        n = static_cast<long long>((limit - static_cast<double>(over)) / static_cast<double>(w));
        n = n < 0 ? 0 : n;
        while (n > 0 && static_cast<double>(over + static_cast<u64>(n - 1) * w) >= limit) --n;
        while (n < V && static_cast<double>(over + static_cast<u64>(n) * w) < limit) ++n;
      }
      ties = n < ties ? n : ties;
    }
  }
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  const double least = mp > 0.f ? static_cast<double>(fminf(mp, 1.f)) * kOne : 0.0;

  // mass and ties of 32 equal parts of the vocabulary, one per warp
  const u64 border_w = static_cast<double>(weigh(border)) >= least ? weigh(border) : 0;
  const int part = ((V + kWarps - 1) / kWarps + 31) / 32 * 32;
  auto over_mass = [&](uint32_t key) -> u64 {
    if (key <= border) return 0;
    const u64 w = weigh(key);
    return static_cast<double>(w) >= least ? w : 0;
  };
  {
    u64 s = 0;
    int c = 0;
    for (int i = warp * part + lane; i < min(V, (warp + 1) * part); i += 32) {
      const uint32_t key = key_of(load_logit(x, i));
      s += over_mass(key);
      c += key == border;
    }
    s = warp_sum(s);
    c = warp_sum(c);
    if (lane == 0) {
      seg_mass[warp] = s;
      seg_ties[warp] = c;
    }
  }
  __syncthreads();
  u64 total = 0, before = 0;
  long long ties_before = 0;
  int at_part = -1;
  {
    long long t = 0;
    for (int s = 0; s < kWarps; ++s) {
      const long long left = ties - t;
      const long long kept = left < 0 ? 0 : (left < seg_ties[s] ? left : seg_ties[s]);
      total += seg_mass[s] + static_cast<u64>(kept) * border_w;
      t += seg_ties[s];
    }
  }
  const float uf = a.u[row];
  const double u = uf > 0.f ? static_cast<double>(fminf(uf, 0.99999994f)) : 0.0;
  const double target = u * static_cast<double>(total);
  {
    u64 sum = 0;
    long long t = 0;
    for (int s = 0; s < kWarps; ++s) {
      const long long left = ties - t;
      const long long kept = left < 0 ? 0 : (left < seg_ties[s] ? left : seg_ties[s]);
      const u64 m = seg_mass[s] + static_cast<u64>(kept) * border_w;
      if (at_part < 0 && static_cast<double>(sum + m) > target) {
        at_part = s;
        before = sum;
        ties_before = t;
      }
      sum += m;
      t += seg_ties[s];
    }
  }
  // the token's part once more, kThreads tokens at a time
  if (tid == 0) s_token = V;
  __syncthreads();
  for (int i0 = at_part * part; i0 < min(V, (at_part + 1) * part); i0 += kThreads) {
    const int i = i0 + tid;
    const bool in = i < min(V, (at_part + 1) * part);
    const uint32_t key = in ? key_of(load_logit(x, i)) : 0;
    int n_ties;
    const int tie = block_scan(static_cast<int>(in && key == border), red_c, n_ties);
    u64 w = in ? over_mass(key) : 0;
    if (in && key == border && ties_before + tie < ties) w = border_w;
    u64 mass;
    const u64 sum = before + block_scan(w, red_m, mass) + w;
    if (w > 0 && static_cast<double>(sum) > target) atomicMin(&s_token, i);
    __syncthreads();
    if (s_token < V) {
      if (i == s_token) {
        a.tokens[row] = i;
        if (a.prob) a.prob[row] = static_cast<float>(weigh.real(key) * kOne / static_cast<double>(total));
      }
      return;
    }
    before += mass;
    ties_before += n_ties;
  }
}

}  // namespace

cudaError_t launch_sample(cudaStream_t st, const SampleArgs& a, int dtype) {
  if (dtype == NLD_F32) sample_kernel<float><<<a.rows, kThreads, 0, st>>>(a);
  else sample_kernel<__nv_bfloat16><<<a.rows, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace nld
