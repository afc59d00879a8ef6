// Block-causal GQA attention over the paged KV cache for wide query tiles (up to 128 rows of a kv head),
// on tcgen05: over the e4m3 cache (nld_attention_q8) and, for both passes of the shared-prefix attention
// (nld_attention_shared), over the bf16 cache.
//
//   o = softmax(q K^T / sqrt(hd) + mask) V;   e4m3: K = k_scale[g] k8,  V = v_scale[g] v8
//
// One CTA per (KV split, kv head, sequence x query tile); row = position * G + head.  128 keys cost 1024
// cycles of tensor core (S = Q K^T and O += P V, 128 x 128 x 128 each) and as many of the exponential
// unit (16 a cycle and SM), so the two have to run side by side: the even and the odd pages are two
// streams, each with its own S, O, running max and sum, its own four softmax warps (a thread per row) and its
// own issuing thread.  A softmax thread takes its row's 64 scores into registers at once, so S of the stream's
// next page is issued right then and is there when the softmax is done; P (in 16 bits) goes beside it, and O += P V
// runs behind.  That fills tensor memory: 64 columns of S and 32 of P a stream, 128 of O, and 64 of Q.  Q is there
// because shared memory is the next bound: a page's K and V cross it twice (256 cycles in, 256 out to the tensor
// core), and 512 more if Q had to be read for every S.  The streams' partials meet in shared memory at the end,
// those of the KV splits over the cluster's distributed shared memory, in a fixed order.
//
// What it measured (8 sequences of 16416 keys, 32 rows, 32 / 8 heads, e4m3: 98 to 104 us, 0.68 PFLOP/s, at the 1.7 GHz that the
// power limit leaves; 90 for the first 30 ms): two pages of 128 rows take
// 1850 cycles, 55 % of the exponential unit; the rest is the latency of a softmax thread's steps (scores in 85 cycles,
// maximum 175, exponentials 512 to 800, waits 370, P out 100).  Two threads a row (sixteen softmax warps) took 10 to
// 17 % longer, a quarter of the exponentials as polynomials on the multiply-add pipe 1 to 6 %, the next page's scores
// fetched under this one's exponentials 9 %, the maximum taken beside the exponentials of a stale one the same time.
// A CTA's fixed cost is 8 us (Q 2, partials 1, merge 3.5), which few pages a CTA do not hide; without splits or a prefix the
// rows go out from the threads that add the streams (64 sequences x 32 rows over 332 keys 62 -> 49 us).
//
// A prefix pass may have more query tiles than SMs, and then a round of clusters that few of them fill.  Where it costs less,
// it is cut into runs of pages (kRuns): a CTA an SM takes as many pages as any other, across query tiles.  Each tile's part
// goes to the workspace as it lies in shared memory, by a copy beside which the next part starts, and the own pass adds
// the parts of a row in their order.  16 sequences x 32 rows of 40 / 8 heads over 4133 shared and 300 own keys: 97 us in clusters, 84 so;
// 20 x 32 rows of 32 / 8 heads over 6000: 120 -> 100; 64 rows a kv head over 16384, in clusters: 47.
//
// bf16: K and V come by TMA into rings of six pages.  e4m3: K's page goes to the tensor core as it comes (kind::f8f6f4)
// against Q in two e4m3 parts (split_e4m3); V's comes by bulk copies, and four warps turn it into an fp16 tile (exact)
// in the swizzled layout of the descriptors, for P rounded to fp16: 2^11 to 2^15 at the row's maximum, so it has fp16's 11
// bits down to 2^-25 of the largest and is off by 2^-36 of that at most below (as in attention_small.cu).  Converting K
// as well took 95 us with eight warps and 166 with four; by integer operations instead of the cvt, 141 with eight.
// K's place frees when S is done, V's when O is.  Over the bf16 cache P is rounded to bf16.  The maximum that exponents
// refer to moves only when it has grown by 2^8 (e4m3: 2^4, that P stays in fp16), so O is rarely rescaled; sums, maxima
// and O are in fp32.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>
#include <atomic>
#include <mutex>

#include "attn_share.cuh"
#include "common.cuh"

namespace nld {

namespace {

constexpr int kTile = kPage;                 // keys of a tile
constexpr int kTileBytes = kTile * 256;      // K (or V) of a tile in 16 bits: [2 boxes of 64 dims][64 keys][128 B]
constexpr int kBoxBytes = kTileBytes / 2;
constexpr int kRawBytes = kTile * 128;       // the same in e4m3: [64 keys][128 B]
constexpr int kSoftmax = 256;                // threads: two streams of 128, a row each
constexpr float kFar = 1048576.f;            // log2 units: from here on a step is 1/8 and more
constexpr uint64_t kWait = 2000000000ull;

template <typename E>
struct Wide {   // bf16
  static constexpr bool kQ8 = false;
  static constexpr float kShift = 0.f, kMove = 8.f;     // log2 units: P at a new reference, and how far it may rise
  static constexpr int kK = 6, kV = 6, kRaw = 0;        // tiles of K, of V, raw ones of V
  static constexpr int kKBytes = kTileBytes;
  static constexpr int kThreads = kSoftmax + 96;        // two issuing warps, a loading one
};
template <>
struct Wide<__nv_fp8_storage_t> {
  static constexpr bool kQ8 = true;
  static constexpr float kShift = 11.f, kMove = 4.f;
  static constexpr int kK = 6, kV = 4, kRaw = 4;
  static constexpr int kKBytes = kRawBytes;
  static constexpr int kThreads = kSoftmax + 96 + 128;   // and four converting ones
};
template <typename E>
__host__ __device__ constexpr int wide_bytes() {
  return 1024 + Wide<E>::kK * Wide<E>::kKBytes + Wide<E>::kV * kTileBytes + Wide<E>::kRaw * kRawBytes + 512;
}

NLD_DEV void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with e4m3 operands, 32 of K a product, four to a column of A.
NLD_DEV void tc_mma_ts_f8(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of an MN-major operand in 128-byte-swizzled atoms (64 elements of MN x 8 of K): `lbo` bytes
// between 64-element MN blocks, `sbo` between groups of 8 K rows.
NLD_DEV uint64_t desc_mn(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}
NLD_DEV void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Wait for this thread's loads of tensor memory; the registers are operands so that no use moves ahead of it.
NLD_DEV void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
NLD_DEV void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
      "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
NLD_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
NLD_DEV float exp2_hw(float x) {   // relative error about 2^-22; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 numbers worked on by one instruction.
typedef unsigned long long f2;
NLD_DEV f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
NLD_DEV void unpair(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
NLD_DEV f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
NLD_DEV f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <bool kHalf>
NLD_DEV uint32_t pack16(float lo, float hi) {
  if constexpr (kHalf) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
// Four e4m3 values as two fp16 pairs: exact.
NLD_DEV void halves_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// The whole warp's wait: the same answer for every lane.
NLD_DEV bool warp_wait(uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, kWait)); }
// One lane of the (converged) warp.
NLD_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}
// Four numbers below 256 of a row whose largest is 128 or more, as e4m3, and what that leaves of them as e4m3: of bf16's eight
// bits the first takes four, rounded, and the second the rest.  Exact from 2^-9 of the row's largest element on; below, where
// the second is subnormal in steps of 2^-9, off by at most 2^-17 of that element.
NLD_DEV void split_e4m3(const float (&q)[4], uint32_t& hi, uint32_t& lo) {
  hi = lo = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    uint32_t back, none;
    halves_of(h, back, none);
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&back));
    hi |= h << (16 * i);
    lo |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q[2 * i] - b.x, q[2 * i + 1] - b.y), __NV_SATFINITE, __NV_E4M3))
          << (16 * i);
  }
}
NLD_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

NLD_DEV void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)), "r"(smem_u32(src)),
               "r"(bytes)
               : "memory");
}
NLD_DEV void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
NLD_DEV void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }   // the source is free
NLD_DEV void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }             // the copies are done

// Weight of a part of a row whose maximum is m in the sum of parts, M their largest: 0 where the row sees none of its keys
// (its O may hold anything), else the smallest number at least, so that NaN in a V row that it sees comes out.
NLD_DEV float merge_weight(float m, float M) { return m == -INFINITY ? 0.f : fmaxf(exp2f(m - M), 1.4e-45f); }

// Columns of tensor memory.
NLD_DEV constexpr uint32_t s_col_of(int stream) { return stream * 96; }
NLD_DEV constexpr uint32_t p_col_of(int stream) { return stream * 96 + 64; }
NLD_DEV constexpr uint32_t o_col_of(int stream) { return 192 + stream * 128; }
constexpr uint32_t kQCol = 448;

template <typename E, int kShare, bool kRuns>
__global__ void __launch_bounds__(Wide<E>::kThreads, 1)
    attn_wide_kernel(const __grid_constant__ CUtensorMap tmKV, const AttnWideArgs a) {
  using W = Wide<E>;
  constexpr bool kQ8 = W::kQ8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;                          // [kK] tiles
  uint8_t* sV = sK + W::kK * W::kKBytes;       // [kV]
  uint8_t* sRaw = sV + W::kV * kTileBytes;     // [kRaw] of V
  uint64_t* bars = reinterpret_cast<uint64_t*>(sRaw + W::kRaw * kRawBytes);
  uint64_t* k_full = bars;             // [kK] tile of K there
  uint64_t* k_empty = bars + 6;        // [kK] S of the tile done
  uint64_t* v_full = bars + 12;        // [kV]
  uint64_t* v_empty = bars + 18;       // [kV] O += P V of the tile done
  uint64_t* raw_full = bars + 24;      // [kRaw] bytes landed
  uint64_t* raw_empty = bars + 28;     // [kRaw] converted
  uint64_t* s_full = bars + 32;        // [stream] S written
  uint64_t* s_read = bars + 34;        // [stream] S in registers
  uint64_t* p_full = bars + 36;        // [stream] P written
  uint64_t* pv_done = bars + 38;       // [stream] O += P V done
  uint64_t* fin = bars + 44;           // every product done
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 45);
  volatile int* s_abort = reinterpret_cast<volatile int*>(bars + 46);
  int* s_bad = reinterpret_cast<int*>(bars + 47);   // [kRaw] the page is outside the pool

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (uniform for the compiler too)
  const int split = blockIdx.x;
  int g = blockIdx.y;
  const int b = blockIdx.z / a.q_tiles;
  const int all = a.m * a.G;                              // rows of the (sequence, kv head)
  int r0 = (blockIdx.z - b * a.q_tiles) * a.rows, rows = min(a.rows, all - r0);   // of this CTA
  const bool softmax_thr = tid < kSoftmax;
  const bool issue_warp = warp == kSoftmax / 32 || warp == kSoftmax / 32 + 1;
  const bool load_thr = tid == kSoftmax + 64;

  if (tid == 0) {
    for (int i = 0; i < W::kK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < W::kV; ++i) {
      mbar_init(&v_full[i], kQ8 ? 4 : 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < W::kRaw; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_read[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(fin, 2);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmKV);
  }
  if (warp == kSoftmax / 32) {
    tmem_alloc(s_tmem, 512);   // S and P of the streams, O of the streams, Q
    tmem_relinquish();
  }

  int len = 0;
  if constexpr (kShare != kPrefixPass) {
    len = a.lens[b];
    if (len < 0 || len > a.pps * kPage - a.m) {   // keys stay inside the page table row
      if (tid == 0) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
      len = max(0, min(len, a.pps * kPage - a.m));
    }
  }
  // keys that a row sees: [0, seen)
  auto seen_by = [&](int r) {
    if constexpr (kShare == kPrefixPass) return a.key_end;
    return len + min((r / a.G) / a.block_size * a.block_size + a.block_size, a.m);
  };
  const int kv_end = seen_by(r0 + rows - 1);   // the last row sees the most
  const int n_pages = (kv_end + kPage - 1) / kPage;
  const int per = (n_pages + a.S - 1) / a.S;
  int t_lo = split * per;
  int ntile = max(0, min(n_pages, t_lo + per) - t_lo);
  // The prefix pass: pages [at, end) of all its (kv head, query tile, page), a query tile's part at a time.  The
  // rings and the barriers run on from one part to the next: done tiles of the CTA, of each stream.
  unsigned at_page = 0, end_page = 0;
  size_t place = 0;
  int done = 0, done_0 = 0, done_1 = 0, part = 0;
  constexpr bool runs = kShare == kPrefixPass && kRuns;
  if constexpr (runs) {
    at_page = split * a.part.per;
    end_page = min(at_page + a.part.per, static_cast<unsigned>(a.Hkv * a.q_tiles) * n_pages);
  }
  auto next_part = [&] {
    const int u = at_page / static_cast<unsigned>(n_pages);
    g = u / a.q_tiles;
    r0 = (u - g * a.q_tiles) * a.rows;
    rows = min(a.rows, all - r0);
    t_lo = at_page - u * n_pages;
    // (uniform for the compiler too)
    ntile = __shfl_sync(0xffffffffu, min(n_pages - t_lo, static_cast<int>(end_page - at_page)), 0);
    place = static_cast<size_t>(u + split) * 128;
  };
  if constexpr (runs) next_part();

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  int n_issued = 0;   // tiles requested (load_thr)
  const int* table = a.page_table + static_cast<size_t>(b) * a.pps;
  // tile j's K and V (e4m3: both raw) into their stages; false: a wait ran out
  auto request = [&](int j) -> bool {
    const int page = table[t_lo + j];
    const bool bad = page < 0 || page >= a.n_pages;
    if (bad) set_err(a.err, NLD_DEVERR_KV_OVERFLOW);
    j += done;
    const int ks = j % W::kK;
    if (j >= W::kK && !mbar_wait(&k_empty[ks], static_cast<uint32_t>(j / W::kK - 1) & 1u, kWait)) return false;
    // (a page outside the pool: rows outside the tensor, which read as zeros)
    const int k_row = bad ? -kPage : (page * 2 * a.Hkv + g) * kPage;
    mbar_arrive_expect_tx(&k_full[ks], W::kKBytes);
    if constexpr (kQ8) {
      tma_load_2d(sK + ks * W::kKBytes, &tmKV, &k_full[ks], 0, k_row);
    } else {
#pragma unroll
      for (int box = 0; box < 2; ++box) tma_load_2d(sK + ks * kTileBytes + box * kBoxBytes, &tmKV, &k_full[ks], box * 64, k_row);
    }
    const int vs = j % (kQ8 ? W::kRaw : W::kV), vn = j / (kQ8 ? W::kRaw : W::kV);
    if (vn > 0 && !mbar_wait(kQ8 ? &raw_empty[vs] : &v_empty[vs], static_cast<uint32_t>(vn - 1) & 1u, kWait)) {
      mbar_wait(&k_full[ks], static_cast<uint32_t>(j / W::kK) & 1u, kWait);   // the copies in flight land
      return false;
    }
    ++n_issued;
    if constexpr (kQ8) {
      s_bad[vs] = bad;
      mbar_arrive_expect_tx(&raw_full[vs], kRawBytes);
      bulk_load(sRaw + vs * kRawBytes,
                static_cast<const uint8_t*>(a.pool) + ((static_cast<size_t>(bad ? 0 : page) * 2 + 1) * a.Hkv + g) * kRawBytes, kRawBytes,
                &raw_full[vs]);
    } else {
      mbar_arrive_expect_tx(&v_full[vs], kTileBytes);
#pragma unroll
      for (int box = 0; box < 2; ++box)
        tma_load_2d(sV + vs * kTileBytes + box * kBoxBytes, &tmKV, &v_full[vs], box * 64,
                    bad ? -kPage : ((page * 2 + 1) * a.Hkv + g) * kPage);
    }
    return true;
  };
  // e4m3: the first tiles come while Q is laid out (97 -> 95 us; over bf16 pages, without a conversion behind them, the
  // block of 32 with a shared prefix took 104 us that way and 98 without)
  constexpr int kAhead = kQ8 ? W::kRaw : 0;
  bool aborted = false;
  float m_ref, l_sum;
  for (;;) {   // (a part of the prefix pass at a time; else once)
  m_ref = -INFINITY;
  l_sum = 0.f;
  const int ahead = part > 0 ? min(W::kK, ntile) : min(kAhead, ntile);
  if (load_thr)
    for (int j = 0; j < ahead && !aborted; ++j) aborted = !request(j);
  // Q into tensor memory, two dims a column (e4m3: four, of its high and then of its low parts): thread (stream x,
  // row r) writes dims 64 x .. of row r
  const int x = tid >> 7, r = tid & 127;   // softmax threads
  float c = a.scale_log2;                  // the scores' scale to log2 units
  if (softmax_thr) {
    const int row = r0 + r, pos = row / a.G;
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(a.q) +
        ((static_cast<size_t>(b) * a.m + (r < rows ? pos : 0)) * a.Hq + static_cast<size_t>(g) * a.G + (r < rows ? row - pos * a.G : 0)) * 128);
    uint4 v[8];   // dims 64 x ..
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r < rows ? src[8 * x + i] : make_uint4(0, 0, 0, 0);
    if constexpr (kQ8) {
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 o = src[8 * (1 - x) + i];   // the row's other half, for its largest element
        const uint32_t w[8] = {v[i].x, v[i].y, v[i].z, v[i].w, o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
      }
      // 2^(7 - e) brings the largest element into [128, 256); zero and subnormal rows keep e in range
      const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -119), 126);
      const float ks = a.k_scale[g];
      float down = copysignf(__uint_as_float(static_cast<uint32_t>(134 - e) << 23), ks);   // (the scores' scale stays positive)
      if (big == INFINITY) down = NAN;   // (e4m3 has no infinity)
      c = fabsf(ks) * a.scale_log2 * __uint_as_float(static_cast<uint32_t>(120 + e) << 23);
      if (c < FLT_MIN) c = FLT_MIN;   // (0 times a masked score would be NaN)
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint4 o = v[i >> 1];
        const uint32_t w0 = (i & 1) ? o.z : o.x, w1 = (i & 1) ? o.w : o.y;
        const float q[4] = {__uint_as_float(w0 << 16) * down, __uint_as_float(w0 & 0xffff0000u) * down,
                            __uint_as_float(w1 << 16) * down, __uint_as_float(w1 & 0xffff0000u) * down};
        split_e4m3(q, hi[i], lo[i]);
      }
      const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kQCol + x * 16;
      tmem_st16u(at, hi);
      tmem_st16u(at + 32, lo);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[16] = {v[4 * h].x, v[4 * h].y, v[4 * h].z, v[4 * h].w, v[4 * h + 1].x, v[4 * h + 1].y, v[4 * h + 1].z,
                                v[4 * h + 1].w, v[4 * h + 2].x, v[4 * h + 2].y, v[4 * h + 2].z, v[4 * h + 2].w, v[4 * h + 3].x,
                                v[4 * h + 3].y, v[4 * h + 3].z, v[4 * h + 3].w};
        tmem_st16u(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kQCol + x * 32 + h * 16, w);
      }
    }
    tmem_wait_st();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (kShare == kPrefixPass)
    if (part == 0) pdl_launch_dependents();

  if (load_thr) {
    // ---------------------------------------------------------------- loads --
    for (int j = ahead; j < ntile && !aborted; ++j) aborted = !request(j);
    if (aborted) {
      *s_abort = 1;
      set_err(a.err, NLD_DEVERR_TIMEOUT);
    }
  } else if (issue_warp) {
    // ------------------------------------------- products of stream y: tiles y, y + 2, .. --
    // The whole warp walks the loop and one lane issues: the operands of tcgen05.mma are uniform registers, and with
    // a single thread in here each one was moved there anew, 480 cycles for the four products of P V.
    const int y = warp - kSoftmax / 32;
    const bool leader = elect_one();   // the same lane throughout: a commit counts the issuing thread's products
    constexpr uint32_t kKind = kQ8 ? (1u << 4) : (1u << 4) | (1u << 7) | (1u << 10);   // fp32 accumulator; fp16 or bf16
    constexpr uint32_t idS = (kQ8 ? 1u << 4 : kKind) | ((static_cast<uint32_t>(kTile) >> 3) << 17) | ((128u >> 4) << 24);   // (e4m3: 0)
    constexpr uint32_t idO = kKind | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);   // B (V) MN-major
    const int mine = ntile > y ? (ntile - y + 1) / 2 : 0;   // tiles of the stream
    const uint32_t s_col = tmem + s_col_of(y), p_col = tmem + p_col_of(y), o_col = tmem + o_col_of(y);
    const uint64_t k_desc = sdesc_k_sw128(smem_u32(sK)), v_desc = desc_mn(smem_u32(sV), kBoxBytes, 1024);
    const int first = y ? done_1 : done_0;   // tiles of the stream in earlier parts
    int ks = (done + y) % W::kK, kp = ((done + y) / W::kK) & 1, vs = (done + y) % W::kV, vp = ((done + y) / W::kV) & 1;   // stage and parity of the stream's next K and V
    // S of the stream's tile i, once the softmax has read that of tile i - 1
    auto s_step = [&](int i) -> bool {
      if (!warp_wait(&k_full[ks], kp) || (i >= 1 && !warp_wait(&s_read[y], static_cast<uint32_t>(first + i - 1) & 1u))) return false;
      tc_fence_after();
      const uint64_t d = k_desc + ks * (W::kKBytes >> 4);
      if (leader) {
        // 32 bytes of a K row a product; e4m3: the high parts of Q, then the low ones
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t q_col = tmem + kQCol + (part * 4 + kk) * 8;
            if constexpr (kQ8) tc_mma_ts_f8(s_col, q_col, d + 2 * kk, idS, (part > 0 || kk > 0) ? 1u : 0u);
            else tc_mma_ts(s_col, q_col, d + part * (kBoxBytes >> 4) + 2 * kk, idS, (part > 0 || kk > 0) ? 1u : 0u);
          }
        tc_commit(&k_empty[ks]);
        tc_commit(&s_full[y]);
      }
      __syncwarp();
      ks += 2;
      if (ks >= W::kK) {
        ks -= W::kK;
        kp ^= 1;
      }
      return true;
    };
    if (mine > 0) aborted = !s_step(0);
    for (int i = 0; i < mine && !aborted; ++i) {
      if ((i + 1 < mine && !s_step(i + 1)) || !warp_wait(&p_full[y], static_cast<uint32_t>(first + i) & 1u) || !warp_wait(&v_full[vs], vp)) {
        aborted = true;
        break;
      }
      tc_fence_after();
      const uint64_t d = v_desc + vs * (kTileBytes >> 4);
      if (leader) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)   // 16 keys: 8 columns of P
          tc_mma_ts(o_col, p_col + k * 8, d + k * (2048 >> 4), idO, (i > 0 || k > 0) ? 1u : 0u);
        tc_commit(&v_empty[vs]);
        tc_commit(&pv_done[y]);
      }
      __syncwarp();
      vs += 2;
      if (vs >= W::kV) {
        vs -= W::kV;
        vp ^= 1;
      }
    }
    if (aborted && leader) {
      *s_abort = 1;
      set_err(a.err, NLD_DEVERR_TIMEOUT);
    }
    // every product of this warp is done before tensor memory is released
    if (leader) {
      tc_commit(fin);
      mbar_wait(fin, part & 1, kWait);
    }
    __syncwarp();
  } else if (softmax_thr) {
    // ----------------------------------------------------------- softmax of stream x, row r --
    const int seen = r < rows ? seen_by(r0 + r) : 0;
    const uint32_t lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lane + s_col_of(x), p_at = tmem + lane + p_col_of(x), o_at = tmem + lane + o_col_of(x);
    const int mine = ntile > x ? (ntile - x + 1) / 2 : 0;   // tiles of the stream
    const int first = x ? done_1 : done_0;
    for (int i = 0; i < mine; ++i) {
      const int j = x + 2 * i;
      // tcgen05.ld / st are for whole warps: every exit of this loop is taken by the warp together
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[x], static_cast<uint32_t>(first + i) & 1u, kWait))) {
        aborted = true;
        break;
      }
      tc_fence_after();
      uint32_t s[2][32];
      tmem_ld32_nowait(s_at, s[0]);
      tmem_ld32_nowait(s_at + 32, s[1]);
      tmem_wait_ld(s[0]);
      tmem_wait_ld(s[1]);
      tc_fence_before();
      __syncwarp();
      if ((tid & 31) == 0) mbar_arrive(&s_read[x]);
      const int left = seen - (t_lo + j) * kTile;   // keys of the tile that the row sees
      if (!__all_sync(0xffffffffu, left >= kTile)) {
#pragma unroll
        for (int k = 0; k < kTile; ++k)
          if (k >= left) s[k >> 5][k & 31] = 0xff800000u;
      }
      float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < kTile; ++k) t[k & 3] = fmaxf(t[k & 3], __uint_as_float(s[k >> 5][k & 31]));
      float mx = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * c;
      const bool far = fabsf(mx) > kFar && fabsf(mx) < INFINITY;
      // (rounded so that the largest exponent is kShift + kMove at most)
      if constexpr (kQ8) mx = __fadd_ru(mx, -W::kShift);
      const bool move = mx > __fadd_rd(m_ref, W::kMove);
      const bool scale_o = move && m_ref != -INFINITY;
      const bool rare = __any_sync(0xffffffffu, scale_o || far);
      if (rare && __any_sync(0xffffffffu, scale_o)) {   // (i > 0: m_ref was set)
        if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[x], static_cast<uint32_t>(first + i - 1) & 1u, kWait))) {
          aborted = true;
          break;
        }
        tc_fence_after();
        const float alpha = scale_o ? exp2f(m_ref - mx) : 1.f;
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          float o[16];
          uint32_t w[16];
          tmem_ld16(o_at + q * 16, o);
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * alpha);
          tmem_st16u(o_at + q * 16, w);
        }
        tmem_wait_st();
        l_sum *= alpha;
      }
      if (move) m_ref = mx;
      const float nb = m_ref == -INFINITY ? 0.f : -m_ref;
      const f2 c2 = pair(c, c), nb2 = pair(nb, nb);
      f2 ls[2] = {0, 0};
      uint32_t p[2][16];
      if (rare && __any_sync(0xffffffffu, far)) {
        // As below, but scores rounded before the reference is taken off: kept unrounded by the multiply-add, the largest one
        // could lie half a step of fp32 from its rounded self, and its exponential be 0 or infinite.  (Apart from the usual
        // code, whose registers it would move: a branch that changes the scores costs 3 %, this 1 % of a bf16 pass at most.)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float p0 = __uint_as_float(s[h][2 * k]), p1 = __uint_as_float(s[h][2 * k + 1]);
            p0 = exp2_hw(__fmul_rn(p0, c) + nb);
            p1 = exp2_hw(__fmul_rn(p1, c) + nb);
            ls[k & 1] = add2(ls[k & 1], pair(p0, p1));
            p[h][k] = pack16<kQ8>(p0, p1);
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const f2 e2 = fma2(pair(__uint_as_float(s[h][2 * k]), __uint_as_float(s[h][2 * k + 1])), c2, nb2);
            float p0, p1;
            unpair(e2, p0, p1);
            p0 = exp2_hw(p0);
            p1 = exp2_hw(p1);
            ls[k & 1] = add2(ls[k & 1], pair(p0, p1));
            p[h][k] = pack16<kQ8>(p0, p1);
          }
        }
      }
      // P is free once O += P V of the tile before has read it
      if (i >= 1 && !__all_sync(0xffffffffu, mbar_wait(&pv_done[x], static_cast<uint32_t>(first + i - 1) & 1u, kWait))) {
        aborted = true;
        break;
      }
      tc_fence_after();
      tmem_st16u(p_at, p[0]);
      tmem_st16u(p_at + 16, p[1]);
      float l0, l1;
      unpair(add2(ls[0], ls[1]), l0, l1);
      l_sum += l0 + l1;
      tmem_wait_st();
      if constexpr (!kQ8) {
        // V rows behind the last key: P is 0 there, V may be anything
        const int dead = (t_lo + j + 1) * kTile - kv_end;
        if (dead > 0) {
          const int vs = (done + j) % W::kV;
          if (!__all_sync(0xffffffffu, mbar_wait(&v_full[vs], static_cast<uint32_t>((done + j) / W::kV) & 1u, kWait))) {
            aborted = true;
            break;
          }
          uint8_t* v = sV + vs * kTileBytes + (kTile - dead) * 128;
          for (int e = r; e < dead * 16; e += 128)
            *reinterpret_cast<uint4*>(v + (e & 1) * kBoxBytes + (e >> 1) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async();
        }
      }
      tc_fence_before();
      __syncwarp();
      if ((tid & 31) == 0) mbar_arrive(&p_full[x]);
    }
    if (!aborted && mine > 0 && !__all_sync(0xffffffffu, mbar_wait(&pv_done[x], static_cast<uint32_t>(first + mine - 1) & 1u, kWait)))
      aborted = true;
    if (aborted) {
      *s_abort = 1;
      set_err(a.err, NLD_DEVERR_TIMEOUT);
    }
    tc_fence_after();
  } else if constexpr (kQ8) {
    if (tid >= kSoftmax + 96) {
      // ------------------------------------------------------------- e4m3 to fp16 --
      // 16 rows of V at a time, a thread 16 bytes of one
      const int ct = tid - (kSoftmax + 96), row_of = ct >> 3, ch = ct & 7;
      for (int j = 0; j < ntile && !aborted; ++j) {
        const int st = j % W::kRaw;   // (as many places as raw ones)
        if (!warp_wait(&raw_full[st], static_cast<uint32_t>(j / W::kRaw) & 1u) ||
            (j >= W::kV && !warp_wait(&v_empty[st], static_cast<uint32_t>(j / W::kV - 1) & 1u))) {
          aborted = true;
          break;
        }
        const uint8_t* src = sRaw + st * kRawBytes + ch * 16;
        uint8_t* dst = sV + st * kTileBytes + (ch >> 2) * kBoxBytes;
        const int live = s_bad[st] ? 0 : kv_end - (t_lo + j) * kTile;   // rows behind the last key: zeros
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = u * 16 + row_of;
          uint4 w = *reinterpret_cast<const uint4*>(src + row * 128);
          if (row >= live) w = make_uint4(0, 0, 0, 0);
          uint4 h[2];
          halves_of(w.x, h[0].x, h[0].y);
          halves_of(w.y, h[0].z, h[0].w);
          halves_of(w.z, h[1].x, h[1].y);
          halves_of(w.w, h[1].z, h[1].w);
          // the 32 bytes are chunks 2 ch and 2 ch + 1 of the box; the upper box's lanes store the odd one first,
          // so that eight lanes never meet in a bank
          const int q = (2 * ch) & 7, odd = ch >> 2;
          *reinterpret_cast<uint4*>(dst + row * 128 + (((q + odd) ^ (row & 7)) << 4)) = odd ? h[1] : h[0];
          *reinterpret_cast<uint4*>(dst + row * 128 + (((q + 1 - odd) ^ (row & 7)) << 4)) = odd ? h[0] : h[1];
        }
        fence_proxy_async();
        __syncwarp();
        if ((tid & 31) == 0) {
          mbar_arrive(&v_full[st]);
          mbar_arrive(&raw_empty[st]);
        }
      }
      if (aborted) {
        *s_abort = 1;
        set_err(a.err, NLD_DEVERR_TIMEOUT);
      }
    }
  }

  // ------------------------------------------------------- the streams' partials --
  __syncthreads();   // every product is done; loads too, unless a wait ran out
  if (load_thr && *s_abort) {   // the copies still in flight land before the rings are overlaid
    for (int t = max(0, n_issued - W::kK); t < n_issued; ++t) {
      mbar_wait(&k_full[t % W::kK], static_cast<uint32_t>(t / W::kK) & 1u, kWait);
      if constexpr (kQ8) mbar_wait(&raw_full[t % W::kRaw], static_cast<uint32_t>(t / W::kRaw) & 1u, kWait);
      else mbar_wait(&v_full[t % W::kV], static_cast<uint32_t>(t / W::kV) & 1u, kWait);
    }
  }
  __syncthreads();
  float* sO = reinterpret_cast<float*>(smem);   // [128][128]; float4 s of row r at s ^ (r % 32)
  float2* sML = reinterpret_cast<float2*>(sO + 128 * 128);   // [128] max, sum
  float2* sX = sML + 128;                       // [stream][128] the streams'
  unsigned* sAt = reinterpret_cast<unsigned*>(sX + 256);   // [2][128] places of the prefix's parts, their numbers
  if (softmax_thr) {
    const bool have = ntile > x && !*s_abort;
    sX[tid] = have ? make_float2(m_ref, l_sum) : make_float2(-INFINITY, 0.f);
  }
  __syncthreads();
  // a thread adds dims 64 x .. of both streams' rows r; they are done, then, if there is nothing else to add
  const bool direct = kShare == 0 && a.S == 1;
  if (softmax_thr) {
    const float2 ml0 = sX[r], ml1 = sX[128 + r];
    const float M = fmaxf(ml0.x, ml1.x);
    const float w0 = merge_weight(ml0.x, M), w1 = merge_weight(ml1.x, M);
    // (a stream without a tile has no O)
    const bool take0 = __any_sync(0xffffffffu, w0 != 0.f), take1 = __any_sync(0xffffffffu, w1 != 0.f);
    const uint32_t lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + x * 64;
    const float L = w0 * ml0.y + w1 * ml1.y;
    uint4* out = nullptr;
    float inv = 0.f, vscale = 1.f;
    if constexpr (kQ8) vscale = a.v_scale[g];
    if (direct && r < rows) {
      const int row = r0 + r, pos = row / a.G;
      out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                     ((static_cast<size_t>(b) * a.m + pos) * a.Hq + static_cast<size_t>(g) * a.G + (row - pos * a.G)) * 128) +
            8 * x;
      inv = 1.f / L;   // (a row sees its own key at least; NaN comes out)
    }
#pragma unroll 1
    for (int u = 0; u < 2; ++u) {
      uint32_t o0[32], o1[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) o0[k] = o1[k] = 0u;
      if (take0) tmem_ld32_nowait(lane + o_col_of(0) + u * 32, o0);
      if (take1) tmem_ld32_nowait(lane + o_col_of(1) + u * 32, o1);
      tmem_wait_ld(o0);
      tmem_wait_ld(o1);
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w0 != 0.f)
          v = make_float4(__uint_as_float(o0[k]) * w0, __uint_as_float(o0[k + 1]) * w0, __uint_as_float(o0[k + 2]) * w0,
                          __uint_as_float(o0[k + 3]) * w0);
        if (w1 != 0.f)
          v = make_float4(fmaf(__uint_as_float(o1[k]), w1, v.x), fmaf(__uint_as_float(o1[k + 1]), w1, v.y),
                          fmaf(__uint_as_float(o1[k + 2]), w1, v.z), fmaf(__uint_as_float(o1[k + 3]), w1, v.w));
        if (!direct) {
          *reinterpret_cast<float4*>(sO + r * 128 + (((x * 16 + u * 8 + (k >> 2)) ^ (r & 31)) << 2)) = v;
        } else {
          o0[k >> 1] = pack16<false>(v.x * inv * vscale, v.y * inv * vscale);
          o0[(k >> 1) + 1] = pack16<false>(v.z * inv * vscale, v.w * inv * vscale);
        }
      }
      if (direct && out != nullptr)
#pragma unroll
        for (int k = 0; k < 4; ++k) out[4 * u + k] = make_uint4(o0[4 * k], o0[4 * k + 1], o0[4 * k + 2], o0[4 * k + 3]);
    }
    if (x == 0) sML[r] = make_float2(M, L);
    if constexpr (runs) fence_proxy_async();
    if constexpr (kShare == kOwnPass && kRuns)
      if (x == 1 && r < rows) {
        unsigned first;
        sAt[128 + r] = share_places(a.part, g, b * all + r0 + r, first);
        sAt[r] = first;
      }
  }
  tc_fence_before();
  __syncthreads();
  const bool last = !runs || at_page + ntile >= end_page || *s_abort;
  if (last && warp == kSoftmax / 32) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (direct) break;

  if constexpr (runs) {   // a part is left as it lies here, by a copy that only the next part's loads wait for
    if (load_thr) {
      bulk_store(a.part.o + place * 128, sO, 128 * 128 * 4);
      bulk_store(a.part.ml + place, sML, 128 * 8);
      bulk_commit();
      if (last) bulk_wait();
      else bulk_wait_read();
    }
    if (last) break;
    at_page += ntile;
    done = __shfl_sync(0xffffffffu, done + ntile, 0);
    done_0 = __shfl_sync(0xffffffffu, done_0 + (ntile + 1) / 2, 0);
    done_1 = __shfl_sync(0xffffffffu, done_1 + ntile / 2, 0);
    ++part;
    next_part();
    continue;
  }

  // the splits' partials: rank q of the cluster finishes rows q, q + S, .., a warp four at a time (one row at a
  // time, the waits on shared memory of other CTAs and on the prefix's partials were half of a short CTA)
  const int S = a.S;
  if (S > 1) cluster_sync();
  float vscale = 1.f;
  if constexpr (kQ8) vscale = a.v_scale[g];
  if constexpr (kShare == kOwnPass) pdl_wait();   // the prefix pass has written its partials
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int d4 = tid & 31;
  const uint32_t o_base = smem_u32(sO), ml_base = smem_u32(sML);
  constexpr int kRows = 4;
  for (int t0 = warp * kRows; rank + t0 * S < rows; t0 += W::kThreads / 32 * kRows) {
    size_t at[kRows], pre_at[kRows];   // token x query head; the prefix's first part
    int pre_n[kRows];
    float2 ml[kRows], pre_ml[kRows];
    float4 acc[kRows], pre[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int rr = min(rank + (t0 + i) * S, rows - 1);   // (past the end: the last row again, not stored)
      const int row = r0 + rr, pos = row / a.G;
      at[i] = (static_cast<size_t>(b) * a.m + pos) * a.Hq + static_cast<size_t>(g) * a.G + (row - pos * a.G);
      // (max, sum) of split q in lane q
      ml[i] = d4 < S ? ld_dsmem_f2((S > 1 ? dsmem_addr(ml_base, d4) : ml_base) + rr * 8) : make_float2(-INFINITY, 0.f);
      if constexpr (kShare == kOwnPass)
        if (a.part.o != nullptr) {
          pre_at[i] = kRuns ? sAt[rr] : at[i];
          if constexpr (kRuns) pre_n[i] = sAt[128 + rr];
          pre_ml[i] = a.part.ml[pre_at[i]];
          pre[i] = kRuns ? *share_at(a.part, pre_at[i], d4) : reinterpret_cast<const float4*>(a.part.o)[at[i] * 32 + d4];
        }
      acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float M[kRows], L[kRows], w[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      M[i] = ml[i].x;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) M[i] = fmaxf(M[i], __shfl_xor_sync(0xffffffffu, M[i], off));
      M[i] = __shfl_sync(0xffffffffu, M[i], 0);
      w[i] = merge_weight(ml[i].x, M[i]);
      L[i] = w[i] * ml[i].y;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) L[i] += __shfl_xor_sync(0xffffffffu, L[i], off);
      L[i] = __shfl_sync(0xffffffffu, L[i], 0);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < S) {
        const uint32_t o_peer = S > 1 ? dsmem_addr(o_base, q) : o_base;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int rr = min(rank + (t0 + i) * S, rows - 1);
          const float4 v = ld_dsmem_f4(o_peer + (rr * 128 + ((d4 ^ (rr & 31)) << 2)) * 4);
          const float wq = __shfl_sync(0xffffffffu, w[i], q);
          if (wq != 0.f) {   // (a split without a key of the row may hold anything)
            acc[i].x += wq * v.x;
            acc[i].y += wq * v.y;
            acc[i].z += wq * v.z;
            acc[i].w += wq * v.w;
          }
        }
      }
    if constexpr (kShare == kOwnPass && kRuns) {   // a part of each row at a time
      int most = 1;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        share_add(pre_ml[i], pre[i], M[i], L[i], acc[i]);
        most = max(most, pre_n[i]);
      }
      for (int n = 1; n < most; ++n) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const size_t to = pre_at[i] + min(n, pre_n[i] - 1) * 128;
          pre_ml[i] = a.part.ml[to];
          pre[i] = *share_at(a.part, to, d4);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (n < pre_n[i]) share_add(pre_ml[i], pre[i], M[i], L[i], acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (rank + (t0 + i) * S >= rows) break;
      if constexpr (kShare == kPrefixPass) {
        reinterpret_cast<float4*>(a.part.o)[at[i] * 32 + d4] = acc[i];
        if (d4 == 0) a.part.ml[at[i]] = make_float2(M[i], L[i]);
        continue;
      }
      if constexpr (kShare == kOwnPass)
        if (!kRuns && a.part.o != nullptr) share_add(pre_ml[i], pre[i], M[i], L[i], acc[i]);
      const float k = 1.f / L[i];   // (a row sees its own key at least; NaN comes out)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at[i] * 128 + 4 * d4) =
          make_uint2(pack16<false>(acc[i].x * k * vscale, acc[i].y * k * vscale), pack16<false>(acc[i].z * k * vscale, acc[i].w * k * vscale));
    }
  }
  break;
  }
  if (a.S > 1) cluster_sync();   // peers may still be reading this CTA's shared memory
}

using WideKernel = void (*)(const CUtensorMap, const AttnWideArgs);
// Kinds of kernels: e4m3, own pass, prefix pass; these two with a prefix pass in runs of pages
int kind_of(const AttnWideArgs& a) { return a.share && a.part.per ? a.share + 2 : a.share; }
WideKernel wide_kernel(int kind) {
  switch (kind) {
    case kOwnPass: return attn_wide_kernel<__nv_bfloat16, kOwnPass, false>;
    case kPrefixPass: return attn_wide_kernel<__nv_bfloat16, kPrefixPass, false>;
    case kOwnPass + 2: return attn_wide_kernel<__nv_bfloat16, kOwnPass, true>;
    case kPrefixPass + 2: return attn_wide_kernel<__nv_bfloat16, kPrefixPass, true>;
  }
  return attn_wide_kernel<__nv_fp8_storage_t, 0, false>;
}
int bytes_of(int kind) { return kind ? wide_bytes<__nv_bfloat16>() : wide_bytes<__nv_fp8_storage_t>(); }
int threads_of(int kind) { return kind ? Wide<__nv_bfloat16>::kThreads : Wide<__nv_fp8_storage_t>::kThreads; }
static_assert(6 * kRawBytes + 4 * kTileBytes >= (128 * 128 + 256) * 4, "the partials overlay the rings");

// Clusters of S CTAs that can be resident at once (asked once per device and S).
cudaError_t wide_capacity(int kind, int S, int sms, int* n) {
  static int cache[16][5][9];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  int* c = dev < 16 ? &cache[dev][kind][S] : nullptr;
  if (c && *c) {
    *n = *c;
    return cudaSuccess;
  }
  if ((e = cudaFuncSetAttribute(wide_kernel(kind), cudaFuncAttributeMaxDynamicSharedMemorySize, bytes_of(kind))) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S * (sms / S));
  cfg.blockDim = dim3(threads_of(kind));
  cfg.dynamicSmemBytes = bytes_of(kind);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaOccupancyMaxActiveClusters(n, wide_kernel(kind), &cfg)) != cudaSuccess) return e;
  *n = std::max(1, *n);
  if (c) *c = *n;
  return cudaSuccess;
}

}  // namespace

// Query tiles and KV splits of a launch.
cudaError_t attn_wide_plan(int batch, int max_len, int sms, AttnWideArgs& a) {
  const int all = a.m * a.G;
  a.q_tiles = (all + 127) / 128;
  a.rows = (all + a.q_tiles - 1) / a.q_tiles;
  const long long units = static_cast<long long>(batch) * a.q_tiles * a.Hkv;
  const int tiles = (max_len + kTile - 1) / kTile;
  // The fewest rounds of resident clusters times a round's length, a tile 1 and the rest of a CTA 16, without a merge 11
  double best = 0;
  for (int S = 1; S <= 8 && S <= tiles; ++S) {
    int cap = 1;
    const cudaError_t e = wide_capacity(kind_of(a), S, sms, &cap);
    if (e != cudaSuccess) return e;
    const double cost = static_cast<double>((units + cap - 1) / cap) * ((tiles + S - 1) / S + (S == 1 && !a.share ? 11.0 : 16.0));
    if (S == 1 || cost < best) {
      best = cost;
      a.S = S;
    }
  }
  if (a.share == kPrefixPass && units * tiles <= INT32_MAX) {
    // Or runs of pages: their parts' rest is 12 (the next part starts beside it), and the own pass reads more: 10, and 2 for
    // each part of a tile.
    const int ctas = std::min(sms, kShareCtas), run = static_cast<int>((units * tiles + ctas - 1) / ctas);
    if (run + 12.0 * ((run + tiles - 2) / tiles + 1) + 10.0 + 2.0 * tiles / run < best) {
      a.S = 1;
      a.part.per = run;
      a.part.pages = tiles;
      a.part.rows = a.rows;
      a.part.q_tiles = a.q_tiles;
      int n;
      return wide_capacity(kind_of(a), 1, sms, &n);   // (readies the kernel)
    }
  }
  return cudaSuccess;
}

cudaError_t launch_attention_wide(cudaStream_t st, const CUtensorMap* tmKV, const AttnWideArgs& a, int batch, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  const unsigned pages = static_cast<unsigned>(a.Hkv * a.q_tiles) * a.part.pages;
  cfg.gridDim = a.share == kPrefixPass && a.part.per ? dim3((pages + a.part.per - 1) / a.part.per)
                                       : dim3(a.S, a.Hkv, batch * a.q_tiles);
  cfg.blockDim = dim3(threads_of(kind_of(a)));
  cfg.dynamicSmemBytes = bytes_of(kind_of(a));
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
  return cudaLaunchKernelEx(&cfg, wide_kernel(kind_of(a)), *tmKV, a);
}

}  // namespace nld
