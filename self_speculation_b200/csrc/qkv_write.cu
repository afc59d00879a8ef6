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
// another (lens -> page table, lens -> angles).  Squares, norm and rotation are in fp32; the only
// roundings are those to the output types.
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

constexpr int kQkvThreads = 256;
constexpr int kU = 4;   // heads of a thread

// x / sc by its rounded reciprocal and one correction with the exact remainder (Markstein's method: the
// rounded quotient); quotients that saturate, infinities and NaN stay as they are.
NLD_DEV float divide(float x, float sc, float r) {
  const float q = x * r;
  return fabsf(q) < 1024.f ? fmaf(fmaf(-q, sc, x), r, q) : q;
}

template <typename T, typename C, int kHd>
__global__ void __launch_bounds__(kQkvThreads) qkv_write_kernel(const QkvWriteArgs a) {
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
  uint4 gain[2][2];   // q, k
  if (norm) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const T* g = static_cast<const T*>(j ? a.k_gain : a.q_gain) + lane * n;
      gain[j][0] = __ldg(reinterpret_cast<const uint4*>(g));
      gain[j][1] = __ldg(reinterpret_cast<const uint4*>(g + half));
    }
  }
  const long long s = static_cast<long long>(len) + i, p = s + a.position_offset;
  if (s < 0 || s >= static_cast<long long>(a.pps) * kPage || p < 0 || p >= a.rope_rows) {
    if (threadIdx.x % 32 == 0) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
    return;
  }
  const int slot = static_cast<int>(s);
  const int page = a.page_table[static_cast<size_t>(b) * a.pps + (slot >> 6)];
  float2 cs[n];   // cos, sin
  {
    const float4* t = reinterpret_cast<const float4*>(a.rope + static_cast<size_t>(p) * half + lane * n);
#pragma unroll
    for (int e = 0; e < n / 2; ++e) {
      const float4 v = __ldg(t + e);
      cs[2 * e] = make_float2(v.x, v.y);
      cs[2 * e + 1] = make_float2(v.z, v.w);
    }
  }
  if (page < 0 || page >= a.n_pages) {
    if (threadIdx.x % 32 == 0) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
    return;
  }

#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int h = h0 + u * kHeads;
    float x[n], y[n];
    Vec<T>::unpack(lo[u], x);
    Vec<T>::unpack(hi[u], y);
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < n; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
      for (int off = lanes >> 1; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (h < a.Hq + a.Hkv) {
        const float inv = rsqrtf(fmaf(ss, 1.0f / kHd, a.eps));
        const bool is_k = h >= a.Hq;
        float gx[n], gy[n];
        Vec<T>::unpack(is_k ? gain[1][0] : gain[0][0], gx);
        Vec<T>::unpack(is_k ? gain[1][1] : gain[0][1], gy);
#pragma unroll
        for (int e = 0; e < n; ++e) {
          x[e] = x[e] * inv * gx[e];
          y[e] = y[e] * inv * gy[e];
        }
      }
    }
    if (h >= heads) continue;
    if (h < a.Hq + a.Hkv) {
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const float c = x[e], r = y[e];
        x[e] = c * cs[e].x - r * cs[e].y;
        y[e] = r * cs[e].x + c * cs[e].y;
      }
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
