// The shared-prefix attention's part of a row's merge, common to its kernels.
#pragma once

#include "common.cuh"
#include "nld_internal.h"

namespace nld {

// (O, max, sum) of a row with the prefix's (ml, o) taken in.
NLD_DEV void share_add(float2 ml, float4 o, float& M, float& L, float4& acc) {
  const float top = fmaxf(M, ml.x);
  const float w = M == -INFINITY ? 0.f : exp2f(M - top), v = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
  L = w * L + v * ml.y;
  acc = make_float4(w * acc.x + v * o.x, w * acc.y + v * o.y, w * acc.z + v * o.z, w * acc.w + v * o.w);
  M = top;
}

// The parts of a prefix pass in runs of pages, for row R (token x query heads of a kv head) of kv head g: the first's place,
// and how many there are, 128 places apart.
NLD_DEV int share_places(const ShareParts& p, int g, int R, unsigned& first) {
  const unsigned qt = static_cast<unsigned>(R) / p.rows, u = g * p.q_tiles + qt;
  const unsigned c0 = u * p.pages / p.per, c1 = ((u + 1) * p.pages - 1) / p.per;
  first = (u + c0) * 128 + (R - qt * p.rows);
  return static_cast<int>(c1 - c0) + 1;
}
// Dims 4 d4 .. of a place: a part is left as it lay in shared memory, in the order that keeps rows out of each other's banks.
NLD_DEV const float4* share_at(const ShareParts& p, size_t place, int d4) {
  return reinterpret_cast<const float4*>(p.o) + place * 32 + (d4 ^ static_cast<int>(place & 31));
}
NLD_DEV void share_add_runs(const ShareParts& p, int g, int R, int d4, float& M, float& L, float4& acc) {
  unsigned first;
  const int n = share_places(p, g, R, first);
#pragma unroll 4
  for (int i = 0; i < n; ++i) share_add(p.ml[first + i * 128], *share_at(p, first + i * 128, d4), M, L, acc);
}

}  // namespace nld
