// The shared-prefix attention's part of a row's merge, common to its kernels.
#pragma once

#include "common.cuh"

namespace nld {

// (O, max, sum) of a row with the prefix's (ml, o) taken in.
NLD_DEV void share_add(float2 ml, float4 o, float M, float& L, float4& acc) {
  const float top = fmaxf(M, ml.x);
  const float w = M == -INFINITY ? 0.f : exp2f(M - top), v = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
  L = w * L + v * ml.y;
  acc = make_float4(w * acc.x + v * o.x, w * acc.y + v * o.y, w * acc.z + v * o.z, w * acc.w + v * o.w);
}

// The merged (O, max, sum) of row `prow` (token x query head), dims 4 d4 ..  The prefix pass leaves it in
// global memory (true: done with the row); the own pass takes the prefix pass's in.
template <int kShare>
NLD_DEV bool share_merge(float* part_o, float2* part_ml, size_t prow, int d4, float M, float& L, float4& acc) {
  if constexpr (kShare == kPrefixPass) {
    reinterpret_cast<float4*>(part_o)[prow * 32 + d4] = acc;
    if (d4 == 0) part_ml[prow] = make_float2(M, L);
    return true;
  }
  if (part_o == nullptr) return false;   // no prefix
  share_add(part_ml[prow], reinterpret_cast<const float4*>(part_o)[prow * 32 + d4], M, L, acc);
  return false;
}

}  // namespace nld
