// Modified attention scores, shared by the attention kernels:
//   s = scale q.k;  s = cap tanh(s / cap) when cap > 0;  s += slope (j - i)
// with j the key's and i the query's position.  The cap comes first: the
// distance term is not capped.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace cpattn {

struct ScoreMod {
  float cap;  // 0: no cap
  float inv;  // 1 / cap
};

__device__ __forceinline__ ScoreMod score_mod_of(float softcap) {
  ScoreMod m;
  m.cap = softcap;
  m.inv = softcap > 0.f ? 1.f / softcap : 0.f;
  return m;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// tanh(y) to about 2^-20 relative: for |y| < 0.2 the series up to y^7 (the
// next term, 62 y^9 / 2835, is below 6e-8 of y there), else
// 1 - 2 / (e^{2 y} + 1) with the approximate ex2 and reciprocal (2^-22 and
// 2^-23 relative).  Both ends come out as +-1 (e = inf, e = 0).  The hardware's
// own tanh is off by 2^-11 of its result, which the log-sum-exp would show.
__device__ __forceinline__ float tanh_fast(float y) {
  const float y2 = y * y;
  const float series =
      fmaf(y * y2, fmaf(y2, fmaf(y2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), y);
  const float e = ex2_approx(y * (2.f * kLog2e));
  return fabsf(y) < 0.2f ? series : fmaf(-2.f, rcp_approx(e + 1.f), 1.f);
}

// Modified score in the log2 domain from the scaled score x.
__device__ __forceinline__ float mod_score(const ScoreMod& m, float x, float slope, float away) {
  if (m.cap > 0.f) x = m.cap * tanh_fast(x * m.inv);
  return fmaf(slope, away, x) * kLog2e;
}

// Logical position of partner p's stripe slot k.
__device__ __forceinline__ int stripe_pos(int k, int p, int P, int I) {
  if (I == 1) return k * P + p;
  const int run = k / I;
  return (run * P + p) * I + (k - run * I);
}

// Position of query token t of row b: the caller's, or the one kv_len gives (a
// decode row's own key is its last; a multi-token row's tokens follow its
// context; t0 is the row's first token).
__device__ __forceinline__ int query_pos(const PartialArgs& a, int b, int t, int t0) {
  if (a.q_pos != nullptr) return __ldg(a.q_pos + t);
  const int L = __ldg(a.kv_len + b);
  return a.q_pos_own ? L - 1 : L + (t - t0);
}

}  // namespace cpattn
