// Block-causal GQA attention over the paged KV cache for small query tiles: over the e4m3 cache
// (nld_attention_q8), and over the bf16 cache for both passes of the shared-prefix attention
// (nld_attention_shared).
//
//   o = softmax(q K^T / sqrt(hd) + mask) V;   e4m3: K = k_scale[g] k8,  V = v_scale[g] v8
//
// with the mask of attention.cu.  Bound by HBM: 256 (bf16: 512) bytes per key and kv head, read once per
// query tile.  One CTA per (KV split, kv head, sequence) takes all of the up to 32 query rows, row =
// position * G + head, so the G heads of a kv head share its K and V.  Its 4 warps are kMT (1 or 2) tiles of 16
// rows x 4 / kMT key groups; a warp walks its own pages with an online softmax of its own, kStages
// steps of 8 KB in flight through shared memory by cp.async: a step's K rows are 4 KB in a row, and so are its
// V rows.  The fragments of mma.sync come from there 16 bytes a lane, which works because the order of the
// summed index of a product is free:
//   S = Q K^T: a lane's 16 bytes of a key row feed four (bf16: two) k16 steps, and Q's fragments are read
//     in the same order;
//   O = P V: a lane takes 16 (bf16: 2 x 8) dims of the four keys that its P fragment holds, one dim
//     per n8 tile; pairs of keys are interleaved by byte permutes.
// e4m3 is exact in fp16, so its products run in fp16 with fp32 accumulators: Q's rows are scaled by
// a power of two into fp16's range (bf16's 8 significant bits fit its 11; what falls below 2^-24 of
// the row's largest element rounds at that size, far under fp32's own error of the sum), P is
// rounded to fp16: half a step is 2^-11 of it, an eighth of the output's own bf16 rounding.  P is 2^15 at the row's
// maximum (the division by the sum takes that out), so it keeps all its bits down to 2^-29 of the largest and is off
// by 2^-40 of that at most below; with 1 there it would be 2^-14 and 2^-25, which many keys of a long cache add up.
// Over the bf16 cache Q goes in as it is and P is rounded to bf16, as in attention.cu.  Maxima, sums and O stay
// in fp32.  Both scales are applied to fp32 values: k_scale within the score's scale, v_scale at the end.
//
// 64 sequences of 1024..8192 keys, 32 / 8 heads, one row each: 124 us for 622 MB (5.0 TB/s); copies laid out by
// fragment instead of by row 155, direct loads into registers 193; 3 or 4 steps in flight with 2 CTAs an SM
// the same 125, twice the splits 131.
//
// The partials (O, max, sum) of a CTA's key groups merge in its shared memory, those of a
// sequence's KV splits over the cluster's distributed shared memory, in a fixed order; the prefix pass of the
// shared-prefix attention leaves the merged partial of a row in global memory, the own pass takes it in.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "attn_share.cuh"
#include "common.cuh"

namespace nld {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 2;         // steps of a warp in flight
constexpr int kStepBytes = 8192;   // of K, then of V, half each
constexpr float kShift = 15.f;     // e4m3: log2 of P at the maximum
constexpr int kRowFloats = 132;    // a partial row in shared memory: 128 dims, max, sum
constexpr int kRing = kWarps * kStages * kStepBytes;   // 64 KB; the partials overlay it
static_assert(kRing >= kWarps * 16 * kRowFloats * 4, "partials");

NLD_DEV void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
NLD_DEV void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 values (the low or high half of w) as an fp16 pair: exact.
NLD_DEV uint32_t half2_of_lo(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}\n" : "=r"(d) : "r"(w));
  return d;
}
NLD_DEV uint32_t half2_of_hi(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}\n" : "=r"(d) : "r"(w));
  return d;
}
NLD_DEV uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
NLD_DEV uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 2^x by the hardware approximation (relative error about 2^-22; 2^-inf = 0).
NLD_DEV float exp2_hw(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 bytes to shared memory, asynchronously; zeros (and no read) where !in.
NLD_DEV void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
NLD_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
NLD_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }
NLD_DEV uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
NLD_DEV uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }


// What a lane reads: for e4m3, with 32 keys a step, K (j, c): 16 dims at 64 c + 16 t of key 8 j + g8, V (jj, i): 16
// dims at 16 g8 of key 16 jj + 2 t + (i & 1) + 8 (i >> 1); for bf16, with 16 keys, K (j, c): 8 dims at 32 c + 8 t of key
// 8 j + g8, V (c, i): 8 dims at 64 c + 8 g8 of key 2 t + (i & 1) + 8 (i >> 1).  Chunk c of row r sits in place c ^ swz(r) of
// its eight, so that neither eight lanes of a K read (two rows, four chunks) nor of a V read (four rows, two
// chunks) meet in a bank.
NLD_DEV int swz(int row) { return (row & 2) | (((row >> 2) ^ row) & 1) << 2; }
template <typename E>
struct Cache;
template <>
struct Cache<__nv_fp8_storage_t> {
  typedef __half Operand;
  static constexpr int kKeys = 32;
};
template <>
struct Cache<__nv_bfloat16> {
  typedef __nv_bfloat16 Operand;
  static constexpr int kKeys = 16;
};

template <int kMT, typename E, int kShare>
__global__ void __launch_bounds__(32 * kWarps, 3) attn_small_kernel(const AttnSmallArgs a) {
  constexpr bool kQ8 = sizeof(E) == 1;
  typedef typename Cache<E>::Operand Operand;
  constexpr int kKeys = Cache<E>::kKeys;          // keys of a step
  constexpr int kSteps = kPage / kKeys;           // steps of a page
  constexpr int kRowBytes = 128 * sizeof(E);
  constexpr int kKW = kWarps / kMT;   // key groups
  extern __shared__ __align__(16) float sm[];   // the ring, then [kWarps][16][kRowFloats] partials
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t = lane & 3;
  const int mt = warp / kKW, kw = warp - mt * kKW;
  const int split = blockIdx.x, g = blockIdx.y;
  const int b = blockIdx.z;
  const int rows = a.m * a.G;   // 16 kMT at most

  int len = 0;
  if constexpr (kShare != kPrefixPass) {
    len = a.lens[b];
    if (len < 0 || len > a.pps * kPage - a.m) {   // keys stay inside the page table row
      if (tid == 0) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
      len = max(0, min(len, a.pps * kPage - a.m));
    }
  }
  // keys that the row's position sees: [0, seen)
  auto seen_by = [&](int r) {
    if constexpr (kShare == kPrefixPass) return a.key_end;
    return len + min((r / a.G) / a.block_size * a.block_size + a.block_size, a.m);
  };
  const int kv_end = seen_by(rows - 1);   // the last row sees the most
  const int n_pages = (kv_end + kPage - 1) / kPage;
  const int per = (n_pages + a.S - 1) / a.S;
  const int pg_lo = split * per, pg_hi = min(n_pages, pg_lo + per);

  // the warp's steps: kSteps of each of its pages, the last page's up to the last key
  const uint8_t* pool = static_cast<const uint8_t*>(a.pool) + static_cast<size_t>(g) * (kPage * kRowBytes);
  const size_t page_bytes = static_cast<size_t>(2) * a.Hkv * kPage * kRowBytes;
  const uint32_t v_off = static_cast<uint32_t>(a.Hkv) * kPage * kRowBytes;
  const int* table = a.page_table + static_cast<size_t>(b) * a.pps;
  const uint32_t ring = smem_u32(sm) + warp * (kStages * kStepBytes);
  int r_pg = pg_lo + kw, r_step = 0;                      // next step to request
  int r_page = r_pg < pg_hi ? table[r_pg] : 0;            // its page, and the page after it
  int r_next = r_pg + kKW < pg_hi ? table[r_pg + kKW] : 0;
  auto request = [&](int stage) {   // one group of copies (an empty one behind the last step)
    if (r_pg < pg_hi) {
      const int j0 = r_pg * kPage + r_step * kKeys;
      const bool bad = r_page < 0 || r_page >= a.n_pages;
      if (bad && lane == 0) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
      const uint8_t* kp = pool + (bad ? 0 : r_page) * page_bytes + r_step * (kKeys * kRowBytes) + lane * 16;
      const uint8_t* vp = kp + v_off;
      // copy i: 512 bytes from row kRowsPer i on
      constexpr int kRowsPer = 512 / kRowBytes;
      const uint32_t dst = ring + stage * kStepBytes;
      const int live = bad ? 0 : kv_end - j0;   // keys past the end are not read: zeros
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = kRowsPer * i + lane / (32 / kRowsPer);
        const uint32_t at = i * 512 + ((lane ^ swz(row)) << 4);
        cp_async16(dst + at, kp + i * 512, row < live);
        cp_async16(dst + kStepBytes / 2 + at, vp + i * 512, row < live);
      }
      if (++r_step == kSteps || j0 + kKeys >= kv_end) {
        r_step = 0;
        r_pg += kKW;
        r_page = r_next;
        r_next = r_pg + kKW < pg_hi ? table[r_pg + kKW] : 0;
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) request(i);
  if constexpr (kShare == kPrefixPass) pdl_launch_dependents();

  // Q fragments; for e4m3 scaled by 2^-e of each row's largest element
  const int ra = mt * 16 + g8, rb = ra + 8;   // rows of the (sequence, kv head)
  const int va = ra < rows ? seen_by(ra) : 0, vb = rb < rows ? seen_by(rb) : 0;
  uint32_t qf[8][4];
  float c_a = a.scale_log2, c_b = a.scale_log2;   // the scores' scale to log2 units
  {
    auto q_row = [&](int r) {
      const int pos = r / a.G;
      return static_cast<const __nv_bfloat16*>(a.q) +
             ((static_cast<size_t>(b) * a.m + pos) * a.Hq + static_cast<size_t>(g) * a.G + (r - pos * a.G)) * 128;
    };
    if constexpr (!kQ8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = h ? rb : ra;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 w = r < rows ? *reinterpret_cast<const uint4*>(q_row(r) + c * 32 + t * 8) : make_uint4(0, 0, 0, 0);
          qf[2 * c][h] = w.x;
          qf[2 * c][2 + h] = w.y;
          qf[2 * c + 1][h] = w.z;
          qf[2 * c + 1][2 + h] = w.w;
        }
      }
    } else {
      float x[2][2][16];   // row, half of the dims, element
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = h ? rb : ra;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
          if (r < rows) {
            w[0] = *reinterpret_cast<const uint4*>(q_row(r) + c * 64 + t * 16);
            w[1] = *reinterpret_cast<const uint4*>(q_row(r) + c * 64 + t * 16 + 8);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t v = word(w[i >> 2], i & 3);
            x[h][c][2 * i] = __uint_as_float(v << 16);
            x[h][c][2 * i + 1] = __uint_as_float(v & 0xffff0000u);
          }
        }
        float big = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) big = fmaxf(big, fabsf(x[h][c][i]));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^-e brings the largest element into [1, 2); zero, subnormal and infinite rows keep e in range
        const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -126), 126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) x[h][c][i] *= down;
        (h ? c_b : c_a) = a.k_scale[g] * a.scale_log2 * up;
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) {   // k16 step s: bytes 4 (s % 4) .. of the lane's chunk s / 4
        const int c = s >> 2, o = (s & 3) * 4;
        qf[s][0] = pack_half2(x[0][c][o], x[0][c][o + 1]);
        qf[s][1] = pack_half2(x[1][c][o], x[1][c][o + 1]);
        qf[s][2] = pack_half2(x[0][c][o + 2], x[0][c][o + 3]);
        qf[s][3] = pack_half2(x[1][c][o + 2], x[1][c][o + 3]);
      }
    }
  }

  float o[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;

  int stage = 0;
  for (int pg = pg_lo + kw; pg < pg_hi; pg += kKW) {
#pragma unroll 1
    for (int hh = 0; hh < kSteps; ++hh) {
      const int j0 = pg * kPage + hh * kKeys;
      if (j0 >= kv_end) break;
      cp_async_wait<kStages - 1>();
      __syncwarp();   // the other lanes' copies have landed too
      const uint32_t src = ring + stage * kStepBytes;
      // S: key j * 8 + g8 of column g8
      constexpr int kJ = kKeys / 8;
      float sc[kJ][4];
#pragma unroll
      for (int j = 0; j < kJ; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
      for (int c = 0; c < 8 / kJ; ++c) {
        uint4 kf[kJ];
#pragma unroll
        for (int j = 0; j < kJ; ++j) kf[j] = lds128(src + (8 * j + g8) * kRowBytes + (((4 * c + t) ^ swz(g8)) << 4));
#pragma unroll
        for (int i = 0; i < (kQ8 ? 4 : 2); ++i)
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            if constexpr (kQ8) {
              const uint32_t w = word(kf[j], i);
              mma_16816(sc[j], qf[4 * c + i], half2_of_lo(w), half2_of_hi(w), Operand());
            } else {
              mma_16816(sc[j], qf[2 * c + i], word(kf[j], 2 * i), word(kf[j], 2 * i + 1), Operand());
            }
          }
      }
      float mx_a = -INFINITY, mx_b = -INFINITY;
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = j0 + j * 8 + 2 * t + e;
          const float s0 = key < va ? sc[j][e] * c_a : -INFINITY;
          const float s1 = key < vb ? sc[j][2 + e] * c_b : -INFINITY;
          sc[j][e] = s0;
          sc[j][2 + e] = s1;
          mx_a = fmaxf(mx_a, s0);
          mx_b = fmaxf(mx_b, s1);
        }
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2));
      mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
      mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2));
      if constexpr (kQ8) {   // the reference, rounded up: P does not exceed 2^kShift
        mx_a = __fadd_ru(mx_a, -kShift);
        mx_b = __fadd_ru(mx_b, -kShift);
      }
      if (__any_sync(0xffffffffu, mx_a > m_a || mx_b > m_b)) {
        const float n_a = fmaxf(m_a, mx_a), n_b = fmaxf(m_b, mx_b);
        // (the first finite maximum of a row scales zeros)
        const float al_a = n_a == m_a ? 1.f : exp2_hw(m_a - n_a), al_b = n_b == m_b ? 1.f : exp2_hw(m_b - n_b);
        m_a = n_a;
        m_b = n_b;
        l_a *= al_a;
        l_b *= al_b;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] *= al_a;
          o[n][1] *= al_a;
          o[n][2] *= al_b;
          o[n][3] *= al_b;
        }
      }
      const float base_a = m_a == -INFINITY ? 0.f : m_a, base_b = m_b == -INFINITY ? 0.f : m_b;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        sc[j][0] = exp2_hw(sc[j][0] - base_a);
        sc[j][1] = exp2_hw(sc[j][1] - base_a);
        sc[j][2] = exp2_hw(sc[j][2] - base_b);
        sc[j][3] = exp2_hw(sc[j][3] - base_b);
        l_a += sc[j][0] + sc[j][1];
        l_b += sc[j][2] + sc[j][3];
      }
      if constexpr (kQ8) {
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          uint32_t p[4];
          p[0] = pack_half2(sc[2 * jj][0], sc[2 * jj][1]);
          p[1] = pack_half2(sc[2 * jj][2], sc[2 * jj][3]);
          p[2] = pack_half2(sc[2 * jj + 1][0], sc[2 * jj + 1][1]);
          p[3] = pack_half2(sc[2 * jj + 1][2], sc[2 * jj + 1][3]);
          uint4 vf[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 16 * jj + 2 * t + (i & 1) + 8 * (i >> 1);
            vf[i] = lds128(src + kStepBytes / 2 + row * kRowBytes + ((g8 ^ swz(row)) << 4));
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {   // dims 16 g8 + 4 w ..
            const uint32_t k0 = word(vf[0], w), k1 = word(vf[1], w), k8 = word(vf[2], w), k9 = word(vf[3], w);
            const uint32_t lo0 = __byte_perm(k0, k1, 0x5140), lo1 = __byte_perm(k0, k1, 0x7362);
            const uint32_t hi0 = __byte_perm(k8, k9, 0x5140), hi1 = __byte_perm(k8, k9, 0x7362);
            mma_16816(o[4 * w], p, half2_of_lo(lo0), half2_of_lo(hi0), Operand());
            mma_16816(o[4 * w + 1], p, half2_of_hi(lo0), half2_of_hi(hi0), Operand());
            mma_16816(o[4 * w + 2], p, half2_of_lo(lo1), half2_of_lo(hi1), Operand());
            mma_16816(o[4 * w + 3], p, half2_of_hi(lo1), half2_of_hi(hi1), Operand());
          }
        }
      } else {
        uint32_t p[4];
        p[0] = pack_bf162(sc[0][0], sc[0][1]);
        p[1] = pack_bf162(sc[0][2], sc[0][3]);
        p[2] = pack_bf162(sc[1][0], sc[1][1]);
        p[3] = pack_bf162(sc[1][2], sc[1][3]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint4 vf[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 2 * t + (i & 1) + 8 * (i >> 1);
            vf[i] = lds128(src + kStepBytes / 2 + row * kRowBytes + (((8 * c + g8) ^ swz(row)) << 4));
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {   // dims 64 c + 8 g8 + 2 w ..
            const uint32_t k0 = word(vf[0], w), k1 = word(vf[1], w), k8 = word(vf[2], w), k9 = word(vf[3], w);
            mma_16816(o[8 * c + 2 * w], p, __byte_perm(k0, k1, 0x5410), __byte_perm(k8, k9, 0x5410), Operand());
            mma_16816(o[8 * c + 2 * w + 1], p, __byte_perm(k0, k1, 0x7632), __byte_perm(k8, k9, 0x7632), Operand());
          }
        }
      }
      __syncwarp();     // every lane has read the step
      request(stage);   // into its place
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
  }
  cp_async_wait<0>();

  l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
  l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
  l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
  l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
  __syncthreads();   // the ring is done with: the partials overlay it
  // the warp's partial: column q = 2 t + e of n tile n is dim 16 q + n, bf16: 64 (n / 8) + 8 q + n % 8
  {
    float* pa = sm + (warp * 16 + g8) * kRowFloats;
    float* pb = pa + 8 * kRowFloats;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int n = 0; n < 16; n += 4) {
        const int d = kQ8 ? 16 * (2 * t + e) + n : 64 * (n >> 3) + 8 * (2 * t + e) + (n & 7);
        *reinterpret_cast<float4*>(pa + d) = make_float4(o[n][e], o[n + 1][e], o[n + 2][e], o[n + 3][e]);
        *reinterpret_cast<float4*>(pb + d) = make_float4(o[n][2 + e], o[n + 1][2 + e], o[n + 2][2 + e], o[n + 3][2 + e]);
      }
    if (t == 0) {
      *reinterpret_cast<float2*>(pa + 128) = make_float2(m_a, l_a);
      *reinterpret_cast<float2*>(pb + 128) = make_float2(m_b, l_b);
    }
  }
  __syncthreads();

  float vs = 1.f;
  if constexpr (kQ8) vs = a.v_scale[g];
  if constexpr (kShare == kOwnPass) pdl_wait();   // the prefix pass has written its partials
  auto store_row = [&](int r, float4 v, float M, float L) {   // dims 4 lane .. of row r, merged
    const int pos = r / a.G;
    const size_t at = (static_cast<size_t>(b) * a.m + pos) * a.Hq + static_cast<size_t>(g) * a.G + (r - pos * a.G);
    if constexpr (kShare == kPrefixPass) {
      reinterpret_cast<float4*>(a.part.o)[at * 32 + lane] = v;
      if (lane == 0) a.part.ml[at] = make_float2(M, L);
      return;
    }
    if constexpr (kShare == kOwnPass)
      if (a.part.o != nullptr) {
        if (a.part.per) share_add_runs(a.part, g, b * rows + r, lane, M, L, v);
        else share_add(a.part.ml[at], reinterpret_cast<const float4*>(a.part.o)[at * 32 + lane], M, L, v);
      }
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + at * 128;
    const float k = 1.f / L;   // a row sees its own key at least
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * k * vs, v.y * k * vs), hi = __floats2bfloat162_rn(v.z * k * vs, v.w * k * vs);
    *reinterpret_cast<uint2*>(dst + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  };
  // one warp per row: the key groups' partials, into the first group's place
  const int S = a.S;
  for (int r = warp; r < rows; r += kWarps) {
    float* first = sm + ((r >> 4) * kKW * 16 + (r & 15)) * kRowFloats;
    float M = -INFINITY;
#pragma unroll
    for (int q = 0; q < kKW; ++q) M = fmaxf(M, first[q * 16 * kRowFloats + 128]);
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < kKW; ++q) {
      const float* p = first + q * 16 * kRowFloats;
      const float w = p[128] == -INFINITY ? 0.f : exp2f(p[128] - M);
      const float4 v = *reinterpret_cast<const float4*>(p + 4 * lane);
      L += w * p[129];
      acc.x += w * v.x;
      acc.y += w * v.y;
      acc.z += w * v.z;
      acc.w += w * v.w;
    }
    if (S == 1) {
      store_row(r, acc, M, L);
    } else {
      __syncwarp();
      *reinterpret_cast<float4*>(first + 4 * lane) = acc;
      if (lane == 0) *reinterpret_cast<float2*>(first + 128) = make_float2(M, L);
    }
  }
  if (S == 1) return;
  cluster_sync();
  // rank q of the cluster finishes rows q, q + S, ..
  const int rank = static_cast<int>(cluster_ctarank());
  const uint32_t base = smem_u32(sm);
  for (int r = rank + warp * S; r < rows; r += S * kWarps) {
    const uint32_t at = ((r >> 4) * kKW * 16 + (r & 15)) * kRowFloats * 4;
    float2 ml[8];
    float4 ov[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      ml[q] = make_float2(-INFINITY, 0.f);
      ov[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q < S) {
        const uint32_t peer = dsmem_addr(base, q) + at;
        ml[q] = ld_dsmem_f2(peer + 128 * 4);
        ov[q] = ld_dsmem_f4(peer + 16 * lane);
      }
    }
    float M = -INFINITY;
#pragma unroll
    for (int q = 0; q < 8; ++q) M = fmaxf(M, ml[q].x);
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (ml[q].x != -INFINITY) {
        const float w = exp2f(ml[q].x - M);
        L += w * ml[q].y;
        acc.x += w * ov[q].x;
        acc.y += w * ov[q].y;
        acc.z += w * ov[q].z;
        acc.w += w * ov[q].w;
      } else {
        L += 0.f * ml[q].y;   // (a split that has met only NaN: no maximum, a sum of NaN)
      }
    }
    store_row(r, acc, M, L);
  }
  cluster_sync();   // peers may still be reading this CTA's shared memory
}

}  // namespace

// 16-row tiles and KV splits of a launch.
void attn_small_plan(int batch, int max_len, int sms, AttnSmallArgs& a) {
  a.mt = a.m * a.G <= 16 ? 1 : 2;
  const int pages = (max_len + kPage - 1) / kPage;
  const long long units = static_cast<long long>(batch) * a.Hkv;
  // splits until every SM holds its three CTAs twice, of a page per key group at least; once beside a prefix, where a
  // sequence's own keys are few (64 sequences of up to 512 keys under one of 16384: 63 -> 55 us for both passes)
  const int kw = kWarps / a.mt;
  long long S = ((a.share == kOwnPass ? 3LL : 6LL) * sms + units - 1) / units;
  S = std::min<long long>(std::min<long long>(S, 8), std::max(1, pages / kw));
  a.S = static_cast<int>(std::max<long long>(1, S));
}

namespace {
using SmallKernel = void (*)(const AttnSmallArgs);
template <typename E, int kShare>
SmallKernel small_kernel(int mt) {
  return mt == 1 ? attn_small_kernel<1, E, kShare> : attn_small_kernel<kSmallRows / 16, E, kShare>;
}
SmallKernel small_kernel(int mt, int share) {
  if (share == kPrefixPass) return small_kernel<__nv_bfloat16, kPrefixPass>(mt);
  if (share == kOwnPass) return small_kernel<__nv_bfloat16, kOwnPass>(mt);
  return small_kernel<__nv_fp8_storage_t, 0>(mt);
}
}  // namespace

cudaError_t launch_attention_small(cudaStream_t st, const AttnSmallArgs& a, int batch, bool pdl) {
  static std::atomic<bool> ready[64];   // per device: the shared-memory limits
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    for (int share : {0, kOwnPass, kPrefixPass})
      for (int mt : {1, 2})
        if ((e = cudaFuncSetAttribute(small_kernel(mt, share), cudaFuncAttributeMaxDynamicSharedMemorySize, kRing)) != cudaSuccess)
          return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.S, a.Hkv, batch);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = kRing;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, small_kernel(a.mt, a.share), a);
}

}  // namespace nld
