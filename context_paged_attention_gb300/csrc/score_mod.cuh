// Modified attention scores, shared by the attention kernels:
//   s = scale q.k;  s = cap tanh(s / cap) when cap > 0;  s += slope (j - i)
// with j the key's and i the query's position.  The cap comes first: the
// distance term is not capped.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace cpattn {

// Kinds of cap: none; up to kPlainCap, where tanh(y) = 1 - 2 / (e^{2 y} + 1)
// with the approximate ex2 and reciprocal (2^-22 and 2^-23 relative) is off by
// at most cap * 2^-21, 3e-5; larger ones, where that error would show in the
// log-sum-exp and |y| < 0.2 takes the series up to y^7 instead (the next term,
// 62 y^9 / 2835, is below 6e-8 of y there): about 2^-20 relative everywhere.
// Both ends come out as +-cap (e = inf, e = 0).  The hardware's own tanh is off
// by 2^-11 of its result.
enum : int { kCapNone = 0, kCapPlain = 1, kCapSeries = 2 };
constexpr float kPlainCap = 64.f;

struct ScoreMod {
  int kind;
  float lin;     // score s of a raw product: s log2 e (no cap), 2 s log2 e / cap (plain), s / cap (series)
  float top;     // cap * log2 e
};

// `scale`: natural-domain score of a raw dot product (descales included)
__device__ __forceinline__ ScoreMod score_mod_of(float softcap, float scale) {
  ScoreMod m;
  m.kind = softcap <= 0.f ? kCapNone : (softcap <= kPlainCap ? kCapPlain : kCapSeries);
  m.top = softcap * kLog2e;
  m.lin = m.kind == kCapNone ? scale * kLog2e : (m.kind == kCapPlain ? 2.f * kLog2e * scale / softcap : scale / softcap);
  return m;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// Capped (or only scaled) score in the log2 domain from the raw product.
template <int KIND>
__device__ __forceinline__ float cap_score(const ScoreMod& m, float raw) {
  const float y = raw * m.lin;
  if constexpr (KIND == kCapNone) return y;
  if constexpr (KIND == kCapPlain) return fmaf(-2.f * m.top, rcp_approx(ex2_approx(y) + 1.f), m.top);
  const float y2 = y * y;
  const float series = fmaf(y * y2, fmaf(y2, fmaf(y2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), y);
  const float e = ex2_approx(y * (2.f * kLog2e));
  return m.top * (fabsf(y) < 0.2f ? series : fmaf(-2.f, rcp_approx(e + 1.f), 1.f));
}

// Modified score in the log2 domain; slope2 = slope * log2 e, away = key's minus query's position.
__device__ __forceinline__ float mod_score(const ScoreMod& m, float raw, float slope2, float away) {
  const float x = m.kind == kCapNone ? cap_score<kCapNone>(m, raw)
                  : m.kind == kCapPlain ? cap_score<kCapPlain>(m, raw) : cap_score<kCapSeries>(m, raw);
  return fmaf(slope2, away, x);
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
