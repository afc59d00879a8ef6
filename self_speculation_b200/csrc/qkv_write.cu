// RMSNorm of every query and key head, rotation by position, and the write of the new K and V
// rows into the paged cache, in one pass over q, k and v (nld_qk_norm_rope).
//
// Per head x of hd elements: y = x / sqrt(mean(x^2) + eps) * gain (q and k, if gains are given),
// then the pairs (i, i + hd/2) turn by the angle of the row's position (rotate-half, the pairing
// of the model's own QKV epilogue):  o_i = y_i c - y_{i+hd/2} s,  o_{i+hd/2} = y_{i+hd/2} c + y_i s.
// V is copied.  K and V rows go to slot len + i of their sequence's pages, as they are or as
// e4m3(x / scale) with one scale per kv head (round to nearest even, saturating at +-448).
//
// Bound by HBM: every element is read once and written once.  A thread holds 16 bytes of the lower
// half of a head and the 16 bytes half a head on, so a rotated pair never leaves its thread and the
// mean takes log2(lanes per head) shuffles; the thread's cos / sin stay in registers for all heads
// of the token that it walks, kU of them loaded at once to keep enough bytes in flight.  Squares,
// norm and rotation are in fp32; the only roundings are those to the output types.
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
constexpr int kU = 4;   // heads a thread loads before it works on the first

template <typename T, typename C>
__global__ void __launch_bounds__(kQkvThreads) qkv_write_kernel(const QkvWriteArgs a) {
  constexpr int n = Vec<T>::n;
  const int half = a.hd >> 1;
  const int lanes = half / n;             // threads per head: 4, 8 or 16
  const int per_tok = lanes * a.groups;
  const long long idx = static_cast<long long>(blockIdx.x) * kQkvThreads + threadIdx.x;
  const long long tok = idx / per_tok;
  const int in_tok = static_cast<int>(idx - tok * per_tok);
  const int group = in_tok / lanes, lane = in_tok - group * lanes;
  const long long M = static_cast<long long>(a.batch) * a.m;
  const int heads = a.Hq + 2 * a.Hkv;

  // every lane of a head has the same token, so the shuffles below stay within live lanes
  bool live = tok < M;
  int b = 0, i = 0, slot = -1, pos = -1, page = -1;
  if (live) {
    b = static_cast<int>(tok / a.m);
    i = static_cast<int>(tok - static_cast<long long>(b) * a.m);
    live = !a.rows || i < a.rows[b];
  }
  if (live) {
    const long long s = static_cast<long long>(a.lens[b]) + i;
    const long long p = s + a.position_offset;
    if (s < 0 || s >= static_cast<long long>(a.pps) * kPage || p < 0 || p >= a.rope_rows) {
      if (in_tok == 0) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
      live = false;
    } else {
      slot = static_cast<int>(s);
      pos = static_cast<int>(p);
      page = a.page_table[static_cast<size_t>(b) * a.pps + (slot >> 6)];
      if (page < 0 || page >= a.n_pages) {
        if (in_tok == 0) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
        live = false;
      }
    }
  }
  float cs[n], sn[n];
#pragma unroll
  for (int e = 0; e < n; ++e) cs[e] = sn[e] = 0.f;
  if (live) {
    const float4* t = reinterpret_cast<const float4*>(a.rope + static_cast<size_t>(pos) * half + lane * n);
#pragma unroll
    for (int e = 0; e < n / 2; ++e) {
      const float4 v = t[e];
      cs[2 * e] = v.x;
      sn[2 * e] = v.y;
      cs[2 * e + 1] = v.z;
      sn[2 * e + 1] = v.w;
    }
  }
  const float inv_hd = 1.0f / static_cast<float>(a.hd);
  const bool norm = a.q_gain != nullptr;

  for (int h0 = 0; h0 < heads; h0 += a.groups * kU) {   // the same trips for every thread
    uint4 lo[kU], hi[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * a.groups + group;
      lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
      if (live && h < heads) {
        const T* src = h < a.Hq ? static_cast<const T*>(a.q) + tok * a.q_ld + static_cast<size_t>(h) * a.hd
                       : h < a.Hq + a.Hkv
                           ? static_cast<const T*>(a.k) + tok * a.k_ld + static_cast<size_t>(h - a.Hq) * a.hd
                           : static_cast<const T*>(a.v) + tok * a.v_ld + static_cast<size_t>(h - a.Hq - a.Hkv) * a.hd;
        lo[u] = *reinterpret_cast<const uint4*>(src + lane * n);
        hi[u] = *reinterpret_cast<const uint4*>(src + half + lane * n);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * a.groups + group;
      float x[n], y[n];
      Vec<T>::unpack(lo[u], x);
      Vec<T>::unpack(hi[u], y);
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < n; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
        for (int off = lanes >> 1; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        if (live && h < a.Hq + a.Hkv) {
          const float inv = rsqrtf(fmaf(ss, inv_hd, a.eps));
          const T* g = static_cast<const T*>(h < a.Hq ? a.q_gain : a.k_gain) + lane * n;
          float gx[n], gy[n];
          Vec<T>::unpack(*reinterpret_cast<const uint4*>(g), gx);
          Vec<T>::unpack(*reinterpret_cast<const uint4*>(g + half), gy);
#pragma unroll
          for (int e = 0; e < n; ++e) {
            x[e] = x[e] * inv * gx[e];
            y[e] = y[e] * inv * gy[e];
          }
        }
      }
      if (!live || h >= heads) continue;
      if (h < a.Hq + a.Hkv) {
#pragma unroll
        for (int e = 0; e < n; ++e) {
          const float p = x[e], r = y[e];
          x[e] = p * cs[e] - r * sn[e];
          y[e] = r * cs[e] + p * sn[e];
        }
      }
      if (h < a.Hq) {
        T* dst = static_cast<T*>(a.q_out) + (tok * a.Hq + h) * a.hd;
        store_vec<n>(dst + lane * n, x);
        store_vec<n>(dst + half + lane * n, y);
      } else {
        const int is_v = h >= a.Hq + a.Hkv;
        const int g = h - a.Hq - (is_v ? a.Hkv : 0);
        if constexpr (sizeof(C) == 1) {
          const float sc = (is_v ? a.v_scale : a.k_scale)[g];
#pragma unroll
          for (int e = 0; e < n; ++e) {
            x[e] = x[e] / sc;
            y[e] = y[e] / sc;
          }
        }
        C* dst = static_cast<C*>(a.pool) +
                 (((static_cast<size_t>(page) * 2 + is_v) * a.Hkv + g) * kPage + (slot & 63)) * a.hd;
        store_vec<n>(dst + lane * n, x);
        store_vec<n>(dst + half + lane * n, y);
      }
    }
  }
}

}  // namespace

cudaError_t launch_qkv_write(cudaStream_t st, QkvWriteArgs a, int dtype, int kv_dtype, int sms) {
  const int lanes = (a.hd / 2) / (dtype == NLD_F32 ? 4 : 8);
  const int heads = a.Hq + 2 * a.Hkv;
  const long long M = static_cast<long long>(a.batch) * a.m;
  // groups of lanes per token: a thread walks heads / groups heads with its cos and sin.  Few tokens:
  // one head per thread, so that the call is one round of loads deep.  Many: kU heads per thread.
  a.groups = heads;
  if (M * heads * lanes > 2LL * sms * kQkvThreads) a.groups = (heads + kU - 1) / kU;
  const long long threads = M * a.groups * lanes;
  const dim3 grid(static_cast<unsigned>((threads + kQkvThreads - 1) / kQkvThreads));
  if (dtype == NLD_F32) {
    if (kv_dtype == NLD_F32) qkv_write_kernel<float, float><<<grid, kQkvThreads, 0, st>>>(a);
    else if (kv_dtype == NLD_BF16) qkv_write_kernel<float, __nv_bfloat16><<<grid, kQkvThreads, 0, st>>>(a);
    else qkv_write_kernel<float, __nv_fp8_storage_t><<<grid, kQkvThreads, 0, st>>>(a);
  } else {
    if (kv_dtype == NLD_F32) qkv_write_kernel<__nv_bfloat16, float><<<grid, kQkvThreads, 0, st>>>(a);
    else if (kv_dtype == NLD_BF16) qkv_write_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kQkvThreads, 0, st>>>(a);
    else qkv_write_kernel<__nv_bfloat16, __nv_fp8_storage_t><<<grid, kQkvThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace nld
