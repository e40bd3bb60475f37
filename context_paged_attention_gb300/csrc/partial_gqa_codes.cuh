// GQA rows of one token over pools of codes: E2M1 (4-bit) pools, and E4M3 pools
// when the scores are modified.
//
// An E2M1 row holds D codes of 4 bits (value 0, 0.5, 1, 1.5, 2, 3, 4 or 6 with a
// sign), an E4M3 scale per 16 values, and the tensor's descale: 72 bytes at
// D 128 where bf16 takes 256 and E4M3 128.  The work split of per-partner calls,
// the partner addressing and the split-KV merge are those of the bf16 decode
// kernel (CTA = chunk of partner p's stripe of row b for KV head h; stripe slot k
// at page k / (page_size / P), slot k % (page_size / P) -- mstar PR #1124
// "Context / Sequence Parallel 1/5", description).  Fused calls are grouped
// differently: a CTA takes every partner's keys of a run of logical pages
// (softmax does not mind the order), so no partner partials are written or
// merged; a row of one run leaves the CTA as final output, longer rows leave
// pieces that the row's last CTA merges.
//
// Heads on the N side of mma.sync m16n8k16, keys (S^T = K Q^T) and dims
// (O^T = V^T P^T) on the M side.  The order of the MMA's k index (dims of S,
// keys of P V) is free as long as both operands follow it, so every lane's
// codes are consecutive in its row and no ldmatrix is needed:
//   K: lane (g = lane / 4, q = lane % 4) reads dims [q D/4, (q + 1) D/4) of
//      keys g and g + 8 with wide loads; the query fragment follows.
//   V: the lane reads dims [g D/8, (g + 1) D/8) of its four keys and pairs the
//      codes of two keys (nibble masks, or byte permutes), so a conversion gives
//      the (key, key') operand pair; at D 128 those are one E2M1 scale block,
//      whose four scales serve all of the lane's m-tiles.
// Codes convert to float16 by cvt (two an instruction); E2M1 codes take their
// scale in float16: at most 2 + 4 significant bits between 2^-10 and 2688, so
// the product is exact.  P is rounded to float16 (relative 2^-11 at most, below
// the bf16 output's 2^-9); its sum and the running max stay in float32.
//
// Loads: cp.async, 16 bytes a lane for the codes and one row's scales a lane,
// stages of 32 keys a warp, two in flight.  With modified scores a warp walks
// its stages from the last key back: scores that fall with the distance then
// meet their maximum first (front to back raised it, and rescaled O, at almost
// every stage); otherwise front to back, which is 3% faster.
// What bounds it: the instructions a key needs (conversion, scale, MMA) more
// than HBM.
#pragma once

#include <type_traits>

#include "gqa_core.cuh"
#include "launch.h"
#include "mma_sync.cuh"
#include "score_mod.cuh"
#include "split_combine.cuh"

namespace cpattn {

namespace {
constexpr int kF4Warps = 4;
constexpr int kF4Keys = 32;    // keys a stage
constexpr int kF4Stages = 2;

template <int D, bool F4>
struct F4Smem {
  static constexpr int ROWB = F4 ? D / 2 : D;   // code bytes of a row
  static constexpr int SCB = F4 ? D / 16 : 0;   // scale bytes of a row
  static constexpr int CODES = kF4Keys * ROWB;
  static constexpr int SCALES = kF4Keys * SCB;
  static constexpr int STAGE = 2 * (CODES + SCALES);
  static constexpr size_t RING = static_cast<size_t>(kF4Warps) * kF4Stages * STAGE;
};

// stage row of MMA key index r (0..7): the permutation spreads the rows that
// one phase of the V loads reads over all banks
__device__ __forceinline__ int f4_row(int r) { return r < 4 ? r : (r ^ 1); }
// position of 16-byte chunk c of stage row r (rows of CH chunks): the same for the K loads' rows
template <int CH>
__device__ __forceinline__ int f4_chunk(int c, int r) {
  return CH == 8 ? c ^ (r & 7) : (CH == 4 ? c ^ (r & 2) : c);
}

template <int BYTES>
__device__ __forceinline__ void cp_async_small(void* dst, const void* src) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(s), "l"(src), "n"(BYTES) : "memory");
}
}  // namespace

// F4: an E2M1 pool, else E4M3.  MOD: modified scores (score_mod.cuh).  E4M3
// rings take 64 KB, three CTAs an SM.
template <int D, int G, bool F4, bool MOD>
__global__ void __launch_bounds__(kF4Warps * 32, G > 8 || !F4 ? 3 : 4) gqa_partial_codes_kernel(const PartialArgs a) {
  using SM = F4Smem<D, F4>;
  constexpr int NW = kF4Warps, KT = kF4Keys, NST = kF4Stages;
  constexpr int CH = SM::ROWB / 16;        // 16-byte chunks of a row's codes
  constexpr int ITERS = KT * CH / 32;
  constexpr int NT = G > 8 ? 2 : 1;        // n-tiles of 8 heads
  constexpr int MMAS = D / 16;             // k-steps of S^T, m-tiles of O^T
  constexpr int KW = SM::ROWB / 16;        // code words a lane holds of a key row
  constexpr int VW = SM::ROWB / 32;        // ... of a value row
  constexpr uint32_t NOROW = 0xffffffffu;  // the launch checks that rows fit 32 bits
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_vmask[NW][NST];
  __shared__ int s_pos[MOD ? NW : 1][MOD ? NST : 1][MOD ? KT : 1];  // positions of a stage's keys

  const int c = blockIdx.x;
  const int p = a.fused ? 0 : blockIdx.y / a.num_kv_heads;  // fused: partners 0 .. P - 1
  const int h = blockIdx.y - p * a.num_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.P;
  const int g8 = lane >> 2, qi = lane & 3;

  pdl_trigger();
  pdl_wait();
  const int b = ordered_row(a.row_order, blockIdx.z, gridDim.z, a.dev_status);
  if (b < 0) return;
  int t = b;
  if (a.qo_indptr != nullptr) {
    t = __ldg(a.qo_indptr + b);
    if (__ldg(a.qo_indptr + b + 1) - t != 1) return;
  }
  int L = __ldg(a.kv_len + b);
  if (L > a.max_kv_len) {
    if (c == 0 && threadIdx.x == 0) report(a.dev_status, CPATTN_DEV_POS_PAST_TABLE);
    L = a.max_kv_len;
  }
  // this CTA's keys: stripe slots [kb, kb + len) of np partners from p on
  int nchunks, kb, len, np;
  if (a.fused) {
    nchunks = max(1, (L + a.run - 1) / a.run);
    // E2M1: whole runs and a rest (64 rows of 512-8192 keys: 81 us, in equal parts 87); E4M3: equal parts
    // (8 rows of 16k-64k: 142 us, whole runs 149)
    const int pages = (L + a.page_size - 1) / a.page_size;
    const int part = F4 ? a.run / a.page_size : (pages + nchunks - 1) / nchunks;
    kb = c * part * a.ps_l;
    len = max(0, min(part, pages - c * part)) * a.ps_l;
    np = P;
  } else {
    const int n_p = stripe_len(L, p, P, a.interleave);
    nchunks = n_p > 0 ? (n_p + a.chunk - 1) / a.chunk : 1;
    kb = c * a.chunk;
    len = max(0, min(n_p - kb, a.chunk));
    np = 1;
  }
  if (c >= nchunks) return;
  const int nstage = (np * len + KT - 1) / KT;
  const int my_n = nstage > warp ? (nstage - warp + NW - 1) / NW : 0;

  // Q as the B operand: head g8 (+ 8), dims q D/4 + 4 m .. + 3 of MMA m
  uint32_t qb[NT][MMAS][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int hd = n * 8 + g8;
    const bool ok = hd < G;
    const uint2* qw = reinterpret_cast<const uint2*>(
        static_cast<const uint8_t*>(a.q) +
        (static_cast<int64_t>(t) * a.num_q_heads + h * G + (ok ? hd : 0)) * (2 * D) + qi * (D / 2));
#pragma unroll
    for (int m = 0; m < MMAS; ++m) {
      const uint2 w = ok ? __ldg(qw + m) : make_uint2(0u, 0u);
      qb[n][m][0] = bf16x2_to_f16x2(w.x);
      qb[n][m][1] = bf16x2_to_f16x2(w.y);
    }
  }

  uint8_t* ring = smem + static_cast<size_t>(warp) * NST * SM::STAGE;
  const uint8_t* poolk = static_cast<const uint8_t*>(a.pool_k);
  const uint8_t* poolv = static_cast<const uint8_t*>(a.pool_v);
  const uint8_t* poolk_lane = poolk + (lane % CH) * 16;  // a lane's chunk of the rows it copies
  const uint8_t* poolv_lane = poolv + (lane % CH) * 16;
  const uint8_t* sclk = poolk + a.scale_off;
  const uint8_t* sclv = poolv + a.scale_off;

  // page ids of the chunk, checked once
  int* spg = reinterpret_cast<int*>(smem + SM::RING);
  const int j0 = kb / a.ps_l;
  if (nstage > 0) {
    const int j1 = (kb + len - 1) / a.ps_l;
    const int pb = __ldg(a.page_indptr + b);
    const int npages = __ldg(a.page_indptr + b + 1) - pb;
    for (int x = threadIdx.x; x <= j1 - j0; x += blockDim.x) {
      const int j = j0 + x;
      int pg = -1;
      if (j >= npages) {
        report(a.dev_status, CPATTN_DEV_POS_PAST_TABLE);
      } else {
        pg = __ldg(a.page_indices + pb + j);
        if (pg < 0 || pg >= a.num_pages) {
          report(a.dev_status, CPATTN_DEV_PAGE_OUT_OF_RANGE);
          pg = -1;
        }
      }
      spg[x] = pg;
    }
  }
  __syncthreads();
  const uint32_t page_rows = static_cast<uint32_t>(a.num_kv_heads) * a.ps_l;
  const uint32_t partner_rows = static_cast<uint32_t>(a.num_pages) * page_rows;
  // the lane's key of the warp's next stage: slot k of partner p + pp
  int pp = 0, k = kb, n_pp = 0;
  if (my_n > 0) {
    const int x0 = (warp + (MOD ? (my_n - 1) * NW : 0)) * KT + lane;
    pp = x0 / len;
    k = kb + x0 - pp * len;
    n_pp = stripe_len(L, p + min(pp, np - 1), P, a.interleave);
  }

  // stage i of this warp: lane = key resolves its row and copies its scales,
  // the codes go 32 consecutive chunks an instruction
  auto issue = [&](int i) {
    if (i < my_n) {
      uint32_t myrow = NOROW;
      if (pp < np && k < n_pp) {
        const int j = page_of_slot(a, k);
        const int pg = spg[j - j0];
        if (pg >= 0)
          myrow = static_cast<uint32_t>(p + pp) * partner_rows + static_cast<uint32_t>(pg) * page_rows +
                  static_cast<uint32_t>(h * a.ps_l + k - j * a.ps_l);
        if constexpr (MOD) s_pos[warp][i % NST][lane] = stripe_pos(k, p + pp, P, a.interleave);
      }
      if constexpr (MOD) {
        k -= NW * KT;
        while (k < kb && pp > 0) {
          k += len;
          --pp;
          n_pp = stripe_len(L, p + min(pp, np - 1), P, a.interleave);
        }
      } else {
        k += NW * KT;
        while (k >= kb + len && pp < np) {
          k -= len;
          ++pp;
          n_pp = stripe_len(L, p + min(pp, np - 1), P, a.interleave);
        }
      }
      const uint32_t vm = __ballot_sync(0xffffffffu, myrow != NOROW);
      if (lane == 0) s_vmask[warp][i % NST] = vm;
      uint8_t* sk = ring + (i % NST) * SM::STAGE;
      uint8_t* sv = sk + SM::CODES;
      uint8_t* ssk = sv + SM::CODES + lane * SM::SCB;
      uint8_t* ssv = ssk + SM::SCALES;
      if constexpr (!F4) {
        // no scales
      } else if (myrow != NOROW) {
        cp_async_small<SM::SCB>(ssk, sclk + static_cast<uint64_t>(myrow) * SM::SCB);
        cp_async_small<SM::SCB>(ssv, sclv + static_cast<uint64_t>(myrow) * SM::SCB);
      } else {  // a masked key's value is 0, never NaN
#pragma unroll
        for (int x = 0; x < SM::SCB; x += 4) *reinterpret_cast<uint32_t*>(ssv + x) = 0u;
      }
#pragma unroll
      for (int it = 0; it < ITERS; ++it) {
        const int idx = it * 32 + lane;
        const int key = idx / CH, ch = idx - key * CH;
        const uint32_t row = __shfl_sync(0xffffffffu, myrow, key);
        const int soff = key * SM::ROWB + f4_chunk<CH>(ch, key) * 16;
        if (row != NOROW) {
          cp_async16(sk + soff, poolk_lane + static_cast<uint64_t>(row) * SM::ROWB);
          cp_async16(sv + soff, poolv_lane + static_cast<uint64_t>(row) * SM::ROWB);
        } else {
          *reinterpret_cast<uint4*>(sv + soff) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
    cp_async_commit();
  };

  float o[NT][MMAS][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int u = 0; u < MMAS; ++u) o[n][u][0] = o[n][u][1] = o[n][u][2] = o[n][u][3] = 0.f;
  float mx[NT][2], l[NT][2];  // heads 8 n + 2 qi, + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
  const float sl = MOD ? 1.f : a.scale * a.k_descale * kLog2e;
  const int krow = f4_row(g8);             // stage rows of keys g8 (+ 8)
  const int vr0 = f4_row(2 * qi), vr1 = f4_row(2 * qi + 1);
  ScoreMod sm_mod;
  float slope[NT][2];
  int qpos = 0;
  if constexpr (MOD) {
    sm_mod = score_mod_of(a.softcap, a.scale * a.k_descale);
    qpos = a.slopes != nullptr ? query_pos(a, b, t, t) : 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hd = n * 8 + 2 * qi + e;
        slope[n][e] = a.slopes != nullptr && hd < G ? __ldg(a.slopes + h * G + hd) * kLog2e : 0.f;
      }
  }

#pragma unroll
  for (int i = 0; i < NST - 1; ++i) issue(i);

  for (int i = 0; i < my_n; ++i) {
    cp_async_wait<NST - 2>();
    __syncwarp();
    issue(i + NST - 1);

    const uint8_t* sk = ring + (i % NST) * SM::STAGE;
    const uint8_t* sv = sk + SM::CODES;
    const uint8_t* ssk = sv + SM::CODES;
    const uint8_t* ssv = ssk + SM::SCALES;
    const uint32_t vm = s_vmask[warp][i % NST];

    // ---- S^T of the two 16-key tiles
    float st[2][NT][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n) st[u][n][0] = st[u][n][1] = st[u][n][2] = st[u][n][3] = 0.f;
      uint32_t kw[2][KW];  // keys g8, g8 + 8: code words
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = u * 16 + e * 8 + krow;
        if constexpr (KW == 2) {
          const uint2 w = *reinterpret_cast<const uint2*>(sk + row * SM::ROWB + qi * 8);
          kw[e][0] = w.x, kw[e][1] = w.y;
        } else {
#pragma unroll
          for (int x = 0; x < KW / 4; ++x) {
            const uint4 w = *reinterpret_cast<const uint4*>(sk + row * SM::ROWB + f4_chunk<CH>(qi * (KW / 4) + x, row) * 16);
            kw[e][4 * x] = w.x, kw[e][4 * x + 1] = w.y, kw[e][4 * x + 2] = w.z, kw[e][4 * x + 3] = w.w;
          }
        }
      }
      if constexpr (F4) {
        uint32_t ks[2][KW / 2];  // one scale a pair of words
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = u * 16 + e * 8 + krow;
          if constexpr (D == 128) {
            const uint32_t s2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ssk + row * SM::SCB + 2 * qi));
            ks[e][0] = __byte_perm(s2, 0u, 0x1010u);
            ks[e][1] = __byte_perm(s2, 0u, 0x3232u);
          } else {
            ks[e][0] = __byte_perm(e4m3x2_to_f16x2(ssk[row * SM::SCB + qi]), 0u, 0x1010u);
          }
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const uint32_t s0 = ks[0][w / 2], s1 = ks[1][w / 2];
          const uint32_t fa[4] = {mul_f16x2(e2m1x2_to_f16x2<0>(kw[0][w]), s0), mul_f16x2(e2m1x2_to_f16x2<0>(kw[1][w]), s1),
                                  mul_f16x2(e2m1x2_to_f16x2<1>(kw[0][w]), s0), mul_f16x2(e2m1x2_to_f16x2<1>(kw[1][w]), s1)};
          const uint32_t fb[4] = {mul_f16x2(e2m1x2_to_f16x2<2>(kw[0][w]), s0), mul_f16x2(e2m1x2_to_f16x2<2>(kw[1][w]), s1),
                                  mul_f16x2(e2m1x2_to_f16x2<3>(kw[0][w]), s0), mul_f16x2(e2m1x2_to_f16x2<3>(kw[1][w]), s1)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(st[u][n], fa, qb[n][2 * w][0], qb[n][2 * w][1]);
            mma_f16(st[u][n], fb, qb[n][2 * w + 1][0], qb[n][2 * w + 1][1]);
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const uint32_t fa[4] = {e4m3x2_to_f16x2(kw[0][w]), e4m3x2_to_f16x2(kw[1][w]), e4m3x2_to_f16x2(kw[0][w] >> 16),
                                  e4m3x2_to_f16x2(kw[1][w] >> 16)};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(st[u][n], fa, qb[n][w][0], qb[n][w][1]);
        }
      }
    }
    // ---- scores in log2 units, masked; the running max over the 32 keys
    const bool full = vm == 0xffffffffu;  // every key of the stage is there
    bool ok[2][2];
    float away[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = u * 16 + e * 8 + krow;
        ok[u][e] = (vm >> r) & 1u;
        if constexpr (MOD)
          away[u][e] = static_cast<float>(s_pos[warp][i % NST][r] - qpos);
      }
    uint32_t pb[2][NT][2];  // P^T as the B operand
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float bm0 = -INFINITY, bm1 = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x0 = st[u][n][2 * e] * sl, x1 = st[u][n][2 * e + 1] * sl;
          if constexpr (MOD) {
            x0 = mod_score(sm_mod, x0, slope[n][0], away[u][e]);
            x1 = mod_score(sm_mod, x1, slope[n][1], away[u][e]);
          }
          if (!full) {
            x0 = ok[u][e] ? x0 : -INFINITY;
            x1 = ok[u][e] ? x1 : -INFINITY;
          }
          st[u][n][2 * e] = x0;
          st[u][n][2 * e + 1] = x1;
          bm0 = fmaxf(bm0, x0);
          bm1 = fmaxf(bm1, x1);
        }
      // the running max is the same in the lanes of a head and rises only when some key exceeds it by more than 8,
      // so the maximum over the lanes is needed only then
      if (__any_sync(0xffffffffu, bm0 > mx[n][0] + 8.f || bm1 > mx[n][1] + 8.f)) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          bm0 = fmaxf(bm0, __shfl_xor_sync(0xffffffffu, bm0, off));
          bm1 = fmaxf(bm1, __shfl_xor_sync(0xffffffffu, bm1, off));
        }
        const bool up0 = bm0 > mx[n][0] + 8.f, up1 = bm1 > mx[n][1] + 8.f;
        const float a0 = up0 ? exp2f(mx[n][0] - bm0) : 1.f;
        const float a1 = up1 ? exp2f(mx[n][1] - bm1) : 1.f;
        if (up0) mx[n][0] = bm0;
        if (up1) mx[n][1] = bm1;
        l[n][0] *= a0;
        l[n][1] *= a1;
#pragma unroll
        for (int u = 0; u < MMAS; ++u) {
          o[n][u][0] *= a0;
          o[n][u][1] *= a1;
          o[n][u][2] *= a0;
          o[n][u][3] *= a1;
        }
      }
      // masked keys: 2^(-inf) = 0; while a head has met no key its max is -inf and 0 stands in
      const float m0 = mx[n][0] == -INFINITY ? 0.f : mx[n][0];
      const float m1 = mx[n][1] == -INFINITY ? 0.f : mx[n][1];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p0 = ex2_approx(st[u][n][2 * e] - m0), p1 = ex2_approx(st[u][n][2 * e + 1] - m1);
          l[n][0] += p0;
          l[n][1] += p1;
          uint32_t tr = pack_f16(p0, p1);
          asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;\n" : "+r"(tr));
          pb[u][n][e] = tr;
        }
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t vw[4][VW];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = u * 16 + (e >> 1) * 8 + ((e & 1) ? vr1 : vr0);
        const uint8_t* src = sv + row * SM::ROWB + f4_chunk<CH>(g8 * VW / 4, row) * 16 + (g8 * VW * 4) % 16;
        if constexpr (VW == 4) {
          const uint4 w = *reinterpret_cast<const uint4*>(src);
          vw[e][0] = w.x, vw[e][1] = w.y, vw[e][2] = w.z, vw[e][3] = w.w;
        } else if constexpr (VW == 2) {
          const uint2 w = *reinterpret_cast<const uint2*>(src);
          vw[e][0] = w.x, vw[e][1] = w.y;
        } else {
          vw[e][0] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
      if constexpr (F4) {
        uint32_t sb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sb[e] = ssv[(u * 16 + (e >> 1) * 8 + ((e & 1) ? vr1 : vr0)) * SM::SCB + (D == 128 ? g8 : g8 >> 1)];
        const uint32_t s01 = e4m3x2_to_f16x2(sb[0] | (sb[1] << 8)), s23 = e4m3x2_to_f16x2(sb[2] | (sb[3] << 8));
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          constexpr uint32_t LO = 0x0f0f0f0fu;
          const uint32_t e01 = (vw[0][w] & LO) | ((vw[1][w] << 4) & ~LO), o01 = ((vw[0][w] >> 4) & LO) | (vw[1][w] & ~LO);
          const uint32_t e23 = (vw[2][w] & LO) | ((vw[3][w] << 4) & ~LO), o23 = ((vw[2][w] >> 4) & LO) | (vw[3][w] & ~LO);
          auto tile = [&](auto ic) {
            constexpr int x = decltype(ic)::value;
            const uint32_t fa[4] = {mul_f16x2(e2m1x2_to_f16x2<x>(e01), s01), mul_f16x2(e2m1x2_to_f16x2<x>(o01), s01),
                                    mul_f16x2(e2m1x2_to_f16x2<x>(e23), s23), mul_f16x2(e2m1x2_to_f16x2<x>(o23), s23)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * w + x], fa, pb[u][n][0], pb[u][n][1]);
          };
          tile(std::integral_constant<int, 0>{});
          tile(std::integral_constant<int, 1>{});
          tile(std::integral_constant<int, 2>{});
          tile(std::integral_constant<int, 3>{});
        }
      } else {
#pragma unroll
        for (int w = 0; w < VW; ++w) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // bytes 2 y, 2 y + 1 of the words: dims 4 w + 2 y, + 1 of the lane's
            const uint32_t sel = y ? 0x7362u : 0x5140u;
            const uint32_t p01 = __byte_perm(vw[0][w], vw[1][w], sel), p23 = __byte_perm(vw[2][w], vw[3][w], sel);
            const uint32_t fa[4] = {e4m3x2_to_f16x2(p01), e4m3x2_to_f16x2(p01 >> 16), e4m3x2_to_f16x2(p23),
                                    e4m3x2_to_f16x2(p23 >> 16)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(o[n][2 * w + y], fa, pb[u][n][0], pb[u][n][1]);
          }
        }
      }
    }
  }
  cp_async_wait<0>();

  // ---- warp states -> shared memory, cross-warp merge
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
  __syncthreads();
  float* sm = reinterpret_cast<float*>(smem);
  float* sm_o = sm;                 // [NW][G][D]
  float* sm_m = sm_o + NW * G * D;  // [NW][G]
  float* sm_l = sm_m + NW * G;      // [NW][G]
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hd = n * 8 + 2 * qi + e;
      if (hd < G) {
        // m-tile u: dims g8 D/8 + 2 u (row g8) and + 1 (row g8 + 8)
        float2* dst = reinterpret_cast<float2*>(sm_o + (warp * G + hd) * D + g8 * (D / 8));
#pragma unroll
        for (int u = 0; u < MMAS; ++u)
          dst[u] = make_float2(o[n][u][e] * a.v_descale, o[n][u][2 + e] * a.v_descale);
        if (g8 == 0) {
          sm_m[warp * G + hd] = mx[n][e];
          sm_l[warp * G + hd] = l[n][e];
        }
      }
    }
  __syncthreads();

  const int64_t orow0 = (static_cast<int64_t>(p) * a.num_tokens + t) * a.num_q_heads + h * G;
  const int64_t slot = (static_cast<int64_t>(t) * P + p) * a.num_kv_heads + h;
  const bool single = (nchunks == 1);
  constexpr int CAP = static_cast<int>(SM::RING / 4);
  for (int idx = threadIdx.x; idx < G * D; idx += blockDim.x) {
    const int g = idx / D;
    const int d = idx - g * D;
    float out, lse;
    merge_stored<D, G>(sm, NW, g, d, out, lse);
    if (a.fused && single) {
      const int64_t hq = static_cast<int64_t>(t) * a.num_q_heads + h * G + g;
      if (a.extra_lse != nullptr) {  // the extra partial merged in
        const float le = __ldg(a.extra_lse + hq);
        const float mm = fmaxf(lse, le);
        if (mm != -INFINITY) {
          const float e0 = expf(lse - mm), e1 = expf(le - mm);
          out = (out * e0 + (e1 != 0.f ? e1 * __ldg(a.extra_o + hq * D + d) : 0.f)) / (e0 + e1);
          lse = mm + logf(e0 + e1);
        }
      }
      if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[hq * D + d] = __float2bfloat16_rn(out);
      else static_cast<float*>(a.out)[hq * D + d] = out;
      if (d == 0 && a.lse_out != nullptr) a.lse_out[hq] = lse;
    } else if (a.fused) {
      const int64_t wrow = ((static_cast<int64_t>(t) * a.num_kv_heads + h) * a.max_runs + c) * G + g;
      a.ws_run_o[wrow * D + d] = out;
      if (d == 0) a.ws_run_lse[wrow] = lse;
    } else if (single) {
      a.o_part[(orow0 + g) * D + d] = out;
      if (d == 0) a.lse_part[lse_slot(a, p, t, h * G + g)] = lse;
    } else {
      const int64_t wrow = (slot * a.max_chunks + c) * G + g;
      a.ws_o[wrow * D + d] = out;
      if (d == 0) a.ws_lse[wrow] = lse;
    }
  }
  if (single) return;
  if (a.fused) {
    int32_t* ticket = a.ws_pair + static_cast<int64_t>(t) * a.num_kv_heads + h;
    if (!take_ticket(ticket, nchunks)) return;
    merge_runs(a, t, 1, h, nchunks, G, D, sm, CAP);
    if (threadIdx.x == 0) *ticket = 0;
  } else {
    if (!take_ticket(a.ws_cnt + slot, nchunks)) return;
    merge_chunks(a, p, h, t, 1, slot, 0, nchunks, G, D, sm, CAP);
    if (threadIdx.x == 0) a.ws_cnt[slot] = 0;
  }
}

template <int D, int G, bool F4, bool MOD>
int launch_codes_t(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  using SM = F4Smem<D, F4>;
  const size_t comb = (static_cast<size_t>(kF4Warps) * G * D + 2 * kF4Warps * G) * sizeof(float);
  const size_t pages = (static_cast<size_t>(a.fused ? a.run / a.page_size : a.chunk / a.ps_l) + 2) * sizeof(int);
  const size_t smem = (SM::RING > comb ? SM::RING : comb) + pages;
  auto kern = gqa_partial_codes_kernel<D, G, F4, MOD>;
  static std::atomic<int> smem_set[64];
  *err = ensure_smem(kern, smem, smem_set);
  if (*err != cudaSuccess) return CPATTN_ERR_CUDA;
  dim3 grid(a.fused ? a.max_runs : a.max_chunks, (a.fused ? 1 : a.P) * a.num_kv_heads, a.qo_indptr != nullptr ? a.num_rows : a.num_tokens);
  *err = launch_pdl(kern, grid, dim3(kF4Warps * 32), smem, s, a);
  return *err == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

template <int D, bool F4, bool MOD>
int codes_dispatch_g(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch_codes_t<D, 1, F4, MOD>(a, s, err);
    case 2: return launch_codes_t<D, 2, F4, MOD>(a, s, err);
    case 4: return launch_codes_t<D, 4, F4, MOD>(a, s, err);
    case 8: return launch_codes_t<D, 8, F4, MOD>(a, s, err);
    case 16: return launch_codes_t<D, 16, F4, MOD>(a, s, err);
    default: return CPATTN_ERR_UNSUPPORTED_SHAPE;
  }
}

template <bool F4, bool MOD>
int codes_dispatch(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  if (a.head_dim == 128) return codes_dispatch_g<128, F4, MOD>(a, s, err);
  if (a.head_dim == 64) return codes_dispatch_g<64, F4, MOD>(a, s, err);
  return CPATTN_ERR_UNSUPPORTED_SHAPE;
}

}  // namespace cpattn
