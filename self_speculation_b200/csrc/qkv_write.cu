// RMSNorm of every query and key head, rotation by position, and the write of the new K and V
// rows into the paged cache, in one pass over q, k and v (nld_qk_norm_rope).
//
// Per head x of hd elements: y = x / sqrt(mean(x^2) + eps) * gain (q and k, if gains are given),
// then the pairs (i, i + hd/2) turn by the angle of the row's position (rotate-half, the pairing
// of the model's own QKV epilogue):  o_i = y_i c - y_{i+hd/2} s,  o_{i+hd/2} = y_{i+hd/2} c + y_i s.
// V is copied.  K and V rows go to slot len + i of their sequence's pages, as they are or as
// e4m3(x / scale) with one scale per kv head (round to nearest even, saturating at +-448).
//
// Bound by HBM: every element is read once and written once.  A warp takes up to kU x (heads per warp)
// heads of one token; a thread holds 16 bytes of the lower half of a head and the 16 bytes half a head
// on, so a rotated pair never leaves its thread and the mean takes log2(lanes per head) shuffles.
// All of a warp's q, k and v are requested before its position, page and angles, which wait on one
// another (lens -> page table, lens -> angles).  Squares, norm and rotation are in fp32, two numbers
// an instruction; the only roundings are those to the output types.
//
// 24 warps an SM (80 registers) and 4 heads a thread measured best: ragged prefill of 8 x 2048 rows of
// 40 + 2 x 8 heads into an e4m3 cache (186 MB) 62 us, 16 warps 75, 28 or 32 warps with spills 68 to 70; 2 heads a thread
// 79; chunks staged through shared memory by cp.async, a persistent warp per token, 87; gains folded into the
// rotation's coefficients, warps of q heads or of k and v heads alone, 66.  The same loads and stores without the
// arithmetic take 40 us: what bounds it is arithmetic and loads that overlap in part.
#include <cuda_fp8.h>

#include "common.cuh"

namespace nld {

namespace {

template <typename T>
struct Vec;   // 16 bytes of T as floats
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static NLD_DEV void unpack(const uint4& r, float* x) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static NLD_DEV void unpack(const uint4& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// n consecutive values to memory in the storage type (n x sizeof(T) bytes, aligned to that up to
// 16 bytes)
template <int n>
NLD_DEV void store_vec(float* p, const float* x) {
#pragma unroll
  for (int i = 0; i < n; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
template <int n>
NLD_DEV void store_vec(__nv_bfloat16* p, const float* x) {
  uint32_t w[n / 2];
#pragma unroll
  for (int i = 0; i < n / 2; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  if constexpr (n == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int n>
NLD_DEV void store_vec(__nv_fp8_storage_t* p, const float* x) {
  uint32_t w[n / 4];
#pragma unroll
  for (int i = 0; i < n / 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  if constexpr (n == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w[0];
}

constexpr int kQkvThreads = 128;
constexpr int kU = 4;   // heads of a thread

// Two fp32 numbers worked on by one instruction.
typedef unsigned long long f2;
NLD_DEV f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
NLD_DEV void split(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
NLD_DEV f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
NLD_DEV f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <typename T>
NLD_DEV void unpack2(const uint4& r, f2 (&x)[Vec<T>::n / 2]) {
  float v[Vec<T>::n];
  Vec<T>::unpack(r, v);
#pragma unroll
  for (int i = 0; i < Vec<T>::n / 2; ++i) x[i] = pair(v[2 * i], v[2 * i + 1]);
}

// x / sc by its rounded reciprocal and one correction with the exact remainder (Markstein's method: the
// rounded quotient); quotients that saturate, infinities and NaN stay as they are.
NLD_DEV float divide(float x, float sc, float r) {
  const float q = x * r;
  return fabsf(q) < 1024.f ? fmaf(fmaf(-q, sc, x), r, q) : q;
}

template <typename T, typename C, int kHd>
__global__ void __launch_bounds__(kQkvThreads, 6) qkv_write_kernel(const QkvWriteArgs a) {
  constexpr int n = Vec<T>::n;
  constexpr int half = kHd / 2;
  constexpr int lanes = half / n;         // threads per head: 4, 8 or 16
  constexpr int kHeads = 32 / lanes;      // heads of a warp at a time
  const unsigned w = blockIdx.x * (kQkvThreads / 32) + threadIdx.x / 32;
  const unsigned tok = w / static_cast<unsigned>(a.groups);
  const int part = static_cast<int>(w - tok * a.groups);
  if (tok >= static_cast<unsigned>(a.batch) * static_cast<unsigned>(a.m)) return;
  const int b = static_cast<int>(tok / static_cast<unsigned>(a.m));
  const int i = static_cast<int>(tok - static_cast<unsigned>(b) * a.m);
  const int lane = threadIdx.x % lanes;
  const int heads = a.Hq + 2 * a.Hkv;
  const int h0 = part * (kHeads * kU) + static_cast<int>(threadIdx.x % 32) / lanes;
  const int len = a.lens[b];
  if (a.rows && i >= a.rows[b]) return;   // the whole warp: padding

  uint4 lo[kU], hi[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int h = h0 + u * kHeads;
    lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
    if (h < heads) {
      const T* src = h < a.Hq ? static_cast<const T*>(a.q) + tok * a.q_ld + h * kHd
                     : h < a.Hq + a.Hkv ? static_cast<const T*>(a.k) + tok * a.k_ld + (h - a.Hq) * kHd
                                        : static_cast<const T*>(a.v) + tok * a.v_ld + (h - a.Hq - a.Hkv) * kHd;
      lo[u] = __ldcs(reinterpret_cast<const uint4*>(src + lane * n));
      hi[u] = __ldcs(reinterpret_cast<const uint4*>(src + half + lane * n));
    }
  }
  const bool norm = a.q_gain != nullptr;
  const long long s = static_cast<long long>(len) + i, p = s + a.position_offset;
  if (s < 0 || s >= static_cast<long long>(a.pps) * kPage || p < 0 || p >= a.rope_rows) {
    if (threadIdx.x % 32 == 0) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
    return;
  }
  const int slot = static_cast<int>(s);
  const int page = a.page_table[static_cast<size_t>(b) * a.pps + (slot >> 6)];
  f2 cs[n / 2], sn[n / 2], ns[n / 2];   // cos, sin, -sin
  {
    const float4* t = reinterpret_cast<const float4*>(a.rope + static_cast<size_t>(p) * half + lane * n);
#pragma unroll
    for (int e = 0; e < n / 2; ++e) {
      const float4 v = __ldg(t + e);
      cs[e] = pair(v.x, v.z);
      sn[e] = pair(v.y, v.w);
      ns[e] = pair(-v.y, -v.w);
    }
  }
  if (page < 0 || page >= a.n_pages) {
    if (threadIdx.x % 32 == 0) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
    return;
  }

#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int h = h0 + u * kHeads;
    f2 x2[n / 2], y2[n / 2];
    unpack2<T>(lo[u], x2);
    unpack2<T>(hi[u], y2);
    if (norm) {
      f2 s2 = mul2(x2[0], x2[0]);
#pragma unroll
      for (int e = 1; e < n / 2; ++e) s2 = fma2(x2[e], x2[e], s2);
#pragma unroll
      for (int e = 0; e < n / 2; ++e) s2 = fma2(y2[e], y2[e], s2);
      float ss, s1;
      split(s2, ss, s1);
      ss += s1;
#pragma unroll
      for (int off = lanes >> 1; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (h < a.Hq + a.Hkv) {
        const float inv = rsqrtf(fmaf(ss, 1.0f / kHd, a.eps));
        const f2 inv2 = pair(inv, inv);
        const T* g = static_cast<const T*>(h < a.Hq ? a.q_gain : a.k_gain) + lane * n;
        f2 g2[n / 2];
        unpack2<T>(__ldg(reinterpret_cast<const uint4*>(g)), g2);
#pragma unroll
        for (int e = 0; e < n / 2; ++e) x2[e] = mul2(mul2(x2[e], inv2), g2[e]);
        unpack2<T>(__ldg(reinterpret_cast<const uint4*>(g + half)), g2);
#pragma unroll
        for (int e = 0; e < n / 2; ++e) y2[e] = mul2(mul2(y2[e], inv2), g2[e]);
      }
    }
    if (h >= heads) continue;
    float x[n], y[n];
#pragma unroll
    for (int e = 0; e < n / 2; ++e) {
      f2 ox = x2[e], oy = y2[e];
      if (h < a.Hq + a.Hkv) {
        ox = fma2(x2[e], cs[e], mul2(y2[e], ns[e]));
        oy = fma2(y2[e], cs[e], mul2(x2[e], sn[e]));
      }
      split(ox, x[2 * e], x[2 * e + 1]);
      split(oy, y[2 * e], y[2 * e + 1]);
    }
    if (h < a.Hq) {
      T* dst = static_cast<T*>(a.q_out) + (static_cast<size_t>(tok) * a.Hq + h) * kHd;
      store_vec<n>(dst + lane * n, x);
      store_vec<n>(dst + half + lane * n, y);
    } else {
      const int is_v = h >= a.Hq + a.Hkv;
      const int g = h - a.Hq - (is_v ? a.Hkv : 0);
      if constexpr (sizeof(C) == 1) {
        const float sc = (is_v ? a.v_scale : a.k_scale)[g];
        if (sc > 1e-37f && sc < 1e37f) {   // (the reciprocal is not subnormal)
          const float r = __frcp_rn(sc);
#pragma unroll
          for (int e = 0; e < n; ++e) {
            x[e] = divide(x[e], sc, r);
            y[e] = divide(y[e], sc, r);
          }
        } else {
#pragma unroll 1
          for (int e = 0; e < n; ++e) {
            x[e] = x[e] / sc;
            y[e] = y[e] / sc;
          }
        }
      }
      C* dst = static_cast<C*>(a.pool) + (((static_cast<size_t>(page) * 2 + is_v) * a.Hkv + g) * kPage + (slot & 63)) * kHd;
      store_vec<n>(dst + lane * n, x);
      store_vec<n>(dst + half + lane * n, y);
    }
  }
}

template <typename T, int kHd>
cudaError_t launch(cudaStream_t st, QkvWriteArgs a, int kv_dtype) {
  constexpr int per = 32 / (kHd / 2 / Vec<T>::n) * kU;   // heads of a warp
  a.groups = (a.Hq + 2 * a.Hkv + per - 1) / per;
  const long long warps = static_cast<long long>(a.batch) * a.m * a.groups;
  const dim3 grid(static_cast<unsigned>((warps + kQkvThreads / 32 - 1) / (kQkvThreads / 32)));
  if (kv_dtype == NLD_F32) qkv_write_kernel<T, float, kHd><<<grid, kQkvThreads, 0, st>>>(a);
  else if (kv_dtype == NLD_BF16) qkv_write_kernel<T, __nv_bfloat16, kHd><<<grid, kQkvThreads, 0, st>>>(a);
  else qkv_write_kernel<T, __nv_fp8_storage_t, kHd><<<grid, kQkvThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qkv_write(cudaStream_t st, const QkvWriteArgs& a, int dtype, int kv_dtype) {
  if (dtype == NLD_F32) return a.hd == 128 ? launch<float, 128>(st, a, kv_dtype) : launch<float, 64>(st, a, kv_dtype);
  return a.hd == 128 ? launch<__nv_bfloat16, 128>(st, a, kv_dtype) : launch<__nv_bfloat16, 64>(st, a, kv_dtype);
}

}  // namespace nld
