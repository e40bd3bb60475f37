// Placement and quantisation of pool rows, shared by the calls that write the
// pool (cp_kv_write, cp_rope_kv_write).
#pragma once

#include "common.cuh"
#include "launch.h"

namespace cpattn {

// E4M3 code of a float32 value, rounded once to the nearest E4M3 value (ties
// to the even code), magnitudes of 448 and more (and infinities) saturated to
// 448, NaN to 0x7F.  Written from the format: normal codes are the float32
// exponent rebiased from 127 to 7 and the mantissa rounded to 3 bits;
// below 2^-6 the codes are the multiples m * 2^-9 (m = 0..8).
__device__ __forceinline__ uint32_t e4m3_rn_satfinite(float x) {
  const uint32_t u = __float_as_uint(x);
  const uint32_t sign = (u >> 24) & 0x80u;
  const float ax = fabsf(x);
  if (ax != ax) return 0x7Fu;
  if (ax >= 448.f) return sign | 0x7Eu;
  if (ax < 0.015625f) return sign | static_cast<uint32_t>(__float2int_rn(ax * 512.f));  // exact scaling
  const uint32_t bits = u & 0x7fffffffu;
  const uint32_t r = (bits + 0x7ffffu + ((bits >> 20) & 1u)) >> 20;  // exponent | 3 mantissa bits, to nearest even
  return sign | (r - ((127u - 7u) << 3));
}

// Value of a non-negative finite E4M3 code (exact).
__device__ __forceinline__ float e4m3_code_value(uint32_t code) {
  const uint32_t e = (code >> 3) & 15u, m = code & 7u;
  return e == 0 ? static_cast<float>(m) * 0.001953125f : __uint_as_float(((e + 120u) << 23) | (m << 20));
}

// Two float32 values -> a byte of E2M1 codes (lo in the low half), nearest
// value, ties to the even code, magnitudes past 6 at 6.
__device__ __forceinline__ uint32_t e2m1x2_rn(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n cvt.u32.u8 %0, b;\n}\n" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// Codes of 8 values v (already x / descale) of a block with scale code `scale`
// (0 where it is 0 or NaN).
__device__ __forceinline__ uint32_t fp4_codes8(const float* v, uint32_t scale) {
  if (scale == 0u || scale == 0x7Fu) return 0u;
  const float s = e4m3_code_value(scale);
  uint32_t codes = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes |= e2m1x2_rn(__fdiv_rn(v[2 * i], s), __fdiv_rn(v[2 * i + 1], s)) << (8 * i);
  return codes;
}

// A block of 16 values of an E2M1 row: its scale is the E4M3 value nearest to
// max |x / descale| / 6, the codes are those of x / descale / scale (IEEE
// quotients, each rounded once).  A block whose scale rounds to 0 (every
// magnitude below 6 * 2^-10 * descale) is stored as zeros; a NaN anywhere
// gives the scale's NaN code, so the whole block reads NaN; an infinity
// saturates its own code at scale 448.
__device__ __forceinline__ void fp4_encode_block(const float (&x)[16], float descale, uint2& codes, uint32_t& scale) {
  float v[16];
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = __fdiv_rn(x[i], descale);
    nan |= v[i] != v[i];
    amax = fmaxf(amax, fabsf(v[i]));
  }
  scale = nan ? 0x7Fu : e4m3_rn_satfinite(__fdiv_rn(amax, 6.f));
  codes = make_uint2(fp4_codes8(v, scale), fp4_codes8(v + 8, scale));
}

// Row b holding token t, or -1 for a padding token (at or past the last
// row's end).  qo_indptr is non-decreasing.
__device__ __forceinline__ int row_of_token(const int32_t* __restrict__ qo_indptr, int num_rows, int t) {
  if (t >= __ldg(qo_indptr + num_rows)) return -1;
  return find_row(qo_indptr, num_rows, t);
}

// Pool row of KV head 0 for position pos of row b (head h is ps_l rows per
// head further), or -1 when the tables do not cover it (recorded if `rep`).
// Offset off of a page goes to partner (off / I) % P, slot
// (off / (I * P)) * I + off % I.
__device__ __forceinline__ int64_t pool_row0(const WriteArgs& a, int b, int pos, bool rep) {
  const int page_idx = pos / a.page_size;
  const int pbeg = __ldg(a.page_indptr + b);
  const int pend = __ldg(a.page_indptr + b + 1);
  if (page_idx >= pend - pbeg) {
    if (rep) report(a.dev_status, CPATTN_DEV_POS_PAST_TABLE);
    return -1;
  }
  const int page = __ldg(a.page_indices + pbeg + page_idx);
  if (page < 0 || page >= a.num_pages) {
    if (rep) report(a.dev_status, CPATTN_DEV_PAGE_OUT_OF_RANGE);
    return -1;
  }
  const int off = pos - page_idx * a.page_size;
  const int run = off / a.interleave;
  const int partner = run % a.P;
  const int slot = (run / a.P) * a.interleave + (off - run * a.interleave);
  const int ps_l = a.page_size / a.P;
  return (static_cast<int64_t>(partner) * a.num_pages + page) * a.num_kv_heads * ps_l + slot;
}

}  // namespace cpattn
