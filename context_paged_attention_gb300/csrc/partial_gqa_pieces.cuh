// Context attention of rows with several query tokens (pieces of prompts, or a
// few drafted tokens) over E2M1 pools, and over any pool with modified scores:
// two 128-row query tiles a CTA on the tcgen05 tensor cores.
//
// Every new token of a row sees the same context (mstar PR #1124 "Context /
// Sequence Parallel 1/5", description: context-only plans), so up to 256 / G
// consecutive tokens of a row and the G heads of KV head h form two dense
// 128-row tiles that share every key:
//   S_t = Q_t K^T  (M = 128 rows of tile t, N = 64 keys, K = head_dim)
//   O_t += P_t V   (N = head_dim, K = 64 keys)
// Why two tiles: a key tile is copied (and for quantised pools converted) once
// for 256 rows, and while the tensor core works for one tile the softmax warps
// of the other keep the exponential and issue slots busy.
//
// Fused calls: one CTA takes all P partners' keys of a run of logical pages,
// 2048 or 4096 positions (softmax does not mind the order: partner 0's slots,
// then partner 1's, ...), so no partner partials leave the SM; items (a block
// of a row's tokens and a head) of more than one run leave normalised pieces in
// the workspace, merged by a second kernel.  Batches of more items than about one a SM are cut
// differently: the cost of all items (from the lengths on the device, so a
// captured call stays balanced) is divided into equal parts, one a CTA, that
// takes whole items and at most two cut ones.  Per-partner calls: one CTA takes
// a chunk of one partner's stripe.
//
// Roles: warps 0-3 and 4-7 own tiles 0 and 1 (thread = query row = TMEM lane:
// online softmax, running max raised only when it grows by more than 8 in log2
// units, P written as 16-bit pairs into tensor memory, from where P V reads
// it; two keys an instruction where the hardware has paired float32
// arithmetic, three where it has a three-way maximum).  Warp 8 issues S, warp 9
// P V: a warp's waits then overlap the other's MMAs.  Warps 10, 11 and 12, 13
// copy 32 keys each of the K and V tiles into rings of 4 and 3 tiles.  bf16
// pools come by cp.async.  E4M3 and E2M1 pools are loaded into registers a tile
// ahead, converted to float16 (exact, block scale included) and stored;
// queries and P are float16 then, so one conversion instruction serves two
// codes (a bf16 target would take three more).  Waiting warps sleep in the
// barrier's own suspended wait: polling took a third of the issue slots.
// (Two threads a row, 16 softmax warps, was slower: half the keys a thread
// with the same waits and barriers, 340 instructions a warp for 32 keys.)
// Tensor memory (512 columns, one CTA an SM), tile t at 256 t: two S buffers of
// 64 columns, O head_dim columns; P of a key tile overwrites the first 32
// columns of its S, so S of the tile after next waits for P V of this one.  Every wait is bounded; one that
// runs out raises the CTA's abort flag, which ends every other wait, and the
// call reports CPATTN_DEV_TC_TIMEOUT.
//
// O is normalised by the float32 sum of the unrounded probabilities: a
// probability is off by 2^-11 (float16) or 2^-8 (bf16) of itself at most.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "mma_sync.cuh"
#include "score_mod.cuh"
#include "split_combine.cuh"
#include "tc05.cuh"
#include "ws_pipe.cuh"

namespace cpattn {

namespace pieces {
constexpr int kTile = 64;       // keys per tile
constexpr int kKStages = 4;
constexpr int kVStages = 3;
constexpr int kMaskSlots = 8;   // masks (and positions) of the tiles in flight
constexpr int kRows = 128;      // query rows of one tile
constexpr int kSoftWarps = 8;
constexpr int kSWarp = 8, kPvWarp = 9;
constexpr int kLoadWarp = 10;   // K: 10, 11, V: 12, 13
constexpr int kUnit = 32;       // keys of a tile that one copy warp takes
constexpr int kUnits = kTile / kUnit;
constexpr int kThreads = 32 * (kLoadWarp + 2 * kUnits);
constexpr int kRun = 2048;      // logical positions of a fused CTA's page run (fewer or twice as many: see launch_t)
constexpr int kSms = 152;
constexpr int kMergeUnroll = 4;
constexpr int kMergeWarps = 4;

// barriers (arrival counts in brackets)
constexpr int B_KFULL = 0;                    // [64 lanes (cp.async) or 2 warps] x4
constexpr int B_KFREE = B_KFULL + kKStages;   // [commit] x4
constexpr int B_VFULL = B_KFREE + kKStages;   // [as K] x3
constexpr int B_VFREE = B_VFULL + kVStages;   // [commit] x3
constexpr int B_SDONE = B_VFREE + kVStages;   // [commit] x2 tiles x2 buffers
constexpr int B_PFULL = B_SDONE + 4;          // [4 warps] x2 x2
constexpr int B_PVDONE = B_PFULL + 4;         // [commit] x2 x2
constexpr int B_Q = B_PVDONE + 4;             // [the softmax warps of the tiles with tokens]
constexpr int B_FIN = B_Q + 1;                // [commit] x2 issuing warps
constexpr int B_COUNT = B_FIN + 2;

template <int D>
struct Layout {
  static constexpr int KB = D / 64;             // 64-column blocks of a row
  static constexpr int QBLK = kRows * 128;
  static constexpr int QTILE = KB * QBLK;
  static constexpr int BLK = kTile * 128;
  static constexpr int TILE = KB * BLK;
  static constexpr uint32_t S_COLS = 64, O_COL = 128, TILE_COLS = 256, TMEM_COLS = 512;
  static constexpr size_t OFF_K = 2 * QTILE;
  static constexpr size_t OFF_V = OFF_K + static_cast<size_t>(kKStages) * TILE;
  static constexpr size_t OFF_BAR = OFF_V + static_cast<size_t>(kVStages) * TILE;
  static constexpr size_t OFF_MASK = OFF_BAR + (B_COUNT * 8 + 15) / 16 * 16;
  static constexpr size_t OFF_POS = OFF_MASK + kMaskSlots * kUnits * 4;
  static constexpr size_t OFF_MISC = OFF_POS + kMaskSlots * kTile * 4;
  static constexpr size_t OFF_PG = OFF_MISC + 16;
  static constexpr int SCRATCH = static_cast<int>(OFF_BAR / 4);  // floats of Q and the rings, free after the loop
  static size_t smem_bytes(int page_slots) { return 1024 + OFF_PG + static_cast<size_t>(page_slots) * 4; }
  static_assert(OFF_POS % 16 == 0, "positions are read 16 bytes at a time");
};

// FMT of the pool
constexpr int kBf16 = 0, kE4m3 = 1, kFp4 = 2;

// Cost of a page for a block with two query tiles or one (a tile's softmax and
// MMAs overlap the other's), and the positions whose time an item's start and
// end take.
constexpr int kCost2 = 5, kCost1 = 3, kStart = 640;

// Where a CTA is in its equal part: row b has ntok tokens from tok0 on and
// `pages` pages; its item (head h, block blk) begins at cost `start`, the CTA
// goes on from page pg0 of it up to cost `end`.  In shared memory between items.
// Piece c of nchunks of the item is pages [pg0, pg1).
struct Place {
  long long start, end, per;
  int b, h, tok0, ntok, pages, blk, pg0, pg1, c, nchunks;
};

// What the walk over rows, heads and blocks needs to know.
struct Walk {
  const int32_t* qo_indptr;
  const int32_t* kv_len;
  int num_rows, num_kv_heads, max_kv_len, page_size, start, qt;

  __device__ bool row(Place& w, int r) const {  // false: the row has fewer than two tokens
    if (r >= num_rows) return false;
    w.b = r;
    w.tok0 = __ldg(qo_indptr + r);
    w.ntok = __ldg(qo_indptr + r + 1) - w.tok0;
    if (w.ntok < 2) return false;
    const long long L = min(__ldg(kv_len + r), max_kv_len);
    w.pages = max(1, static_cast<int>((L + page_size - 1) / page_size));
    return true;
  }
  __device__ int page_cost(const Place& w, int blk) const { return w.ntok - blk * 2 * qt > qt ? kCost2 : kCost1; }
  __device__ long long item_cost(const Place& w, int blk) const {
    return start + static_cast<long long>(w.pages) * page_cost(w, blk);
  }
  __device__ int last_blk(const Place& w) const { return (w.ntok - 1) / (2 * qt); }
  __device__ long long head_cost(const Place& w) const {
    return last_blk(w) * (start + static_cast<long long>(w.pages) * kCost2) + item_cost(w, last_blk(w));
  }
  // The pages of the item that this CTA takes, from pg0 on; false: its part
  // ends before the next one.  A part's border inside an item lies at the page
  // it falls into, so an item's pieces go from the part that reaches the end
  // of its first page to the one that holds its last unit.
  __device__ bool span(Place& w) const {
    const int cost = page_cost(w, w.blk);
    const long long left = w.end - w.start - start;
    w.pg1 = left < cost ? 0 : static_cast<int>(min(static_cast<long long>(w.pages), left / cost));
    const long long first = (w.start + start + cost - 1) / w.per;
    w.c = static_cast<int>(blockIdx.x - first);
    w.nchunks = static_cast<int>((w.start + item_cost(w, w.blk) - 1) / w.per - first) + 1;
    return w.pg1 > w.pg0;
  }
};

// The current item (or run), for its output: piece c of nchunks of head h's
// tokens [s0, s1).
struct Item {
  int c, nchunks, h, s0, s1, ntiles;
};

// E2M1 pools keep a CTA a run: in the loop over items their copy warps, which
// bound that kernel, lose more than the equal parts give (269 us for 253).
__host__ __device__ constexpr bool can_even(int fmt) { return fmt != kFp4; }

struct Geo {
  int run;          // fused: logical positions of a CTA's page run (whole pages)
  int max_runs;     // pieces a row can have (grid.x of a CTA a run)
  int64_t least;    // fused, equal parts: least cost of a part (0: a CTA a run)
  int start;        // cost of an item beside its pages
  float* ws_o;      // fused, several pieces: [T * Hkv][max_runs][G][D]
  float* ws_lse;    // [T * Hkv][max_runs][G]
};

// A value the compiler cannot carry from one loop iteration to the next.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

// 16-bit pair of a P row, and the MMA's operand type
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return F16 ? pack_f16(a, b) : pack_bf16(a, b);
}

// Two float32 values as one operand of the paired instructions.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Modified log2-domain scores of a row's 64 keys, in place (the arithmetic of
// cap_score / mod_score, two keys at a time).
template <int KIND, bool SLOPE>
__device__ __forceinline__ void modify(const ScoreMod& m, float (&sv)[kTile], float slope2, float qpos,
                                       const float4* kp) {
  const uint64_t lin = pair2(m.lin, m.lin), top = pair2(m.top, m.top), ntop = pair2(-2.f * m.top, -2.f * m.top);
  const uint64_t one = pair2(1.f, 1.f), nq = pair2(-qpos, -qpos), sl2 = pair2(slope2, slope2);
#pragma unroll
  for (int e = 0; e < kTile / 4; ++e) {
    float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (SLOPE) k4 = kp[e];  // the same for every row: a broadcast
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float& a = sv[4 * e + 2 * i];
      float& b = sv[4 * e + 2 * i + 1];
      uint64_t x;
      if constexpr (KIND == kCapSeries) {
        x = pair2(cap_score<kCapSeries>(m, a), cap_score<kCapSeries>(m, b));
      } else {
        x = mul2(pair2(a, b), lin);
        if constexpr (KIND == kCapPlain) {
          float u, v;
          unpair2(x, u, v);
          unpair2(add2(pair2(ex2_approx(u), ex2_approx(v)), one), u, v);
          x = fma2(ntop, pair2(rcp_approx(u), rcp_approx(v)), top);
        }
      }
      if (SLOPE) x = fma2(sl2, add2(i ? pair2(k4.z, k4.w) : pair2(k4.x, k4.y), nq), x);
      unpair2(x, a, b);
    }
  }
}

// `bytes` (a multiple of 16) from this CTA's shared memory to global memory, both 16-byte aligned.
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// Bounded wait on a phase that sleeps in the hardware (20 us a try) instead of
// polling; gives up when the abort flag is raised or after some 0.3 s.
__device__ __forceinline__ bool wait_phase(uint32_t mbar, uint32_t parity, const volatile int* abort_flag) {
  for (uint32_t it = 0; it < (1u << 14); ++it) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity), "r"(20000u)
        : "memory");
    if (done) return true;
    if (*abort_flag) return false;
  }
  return false;
}
// The start of this CTA's part; false: it has no page.  (Called, like
// next_place, rather than inlined: the registers of their 64-bit divisions do
// not belong beside the roles' loops.)
static __device__ __noinline__ bool first_place(const Walk walk, int64_t least, Place& place, long long* s_part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Place w;
  long long mine = 0;
  for (int r = tid; r < walk.num_rows; r += kThreads)
    if (walk.row(w, r)) mine += walk.head_cost(w);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_part[warp] = mine;
  if (tid == 0) place.b = -1;
  __syncthreads();
  long long total = 0;
  for (int i = 0; i < kThreads / 32; ++i) total += s_part[i];
  total *= walk.num_kv_heads;
  const long long per = max(static_cast<long long>(least), (total + gridDim.x - 1) / gridDim.x);
  const long long x = blockIdx.x * per;
  if (x >= total) return false;
  // the row that cost x falls into
  long long before = 0;
  for (int r0 = 0; r0 < walk.num_rows; r0 += kThreads) {
    const long long u = walk.row(w, r0 + tid) ? walk.head_cost(w) * walk.num_kv_heads : 0;
    long long incl = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) s_part[warp] = incl;
    __syncthreads();
    long long lo = before + incl - u;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) lo += s_part[i];
      before += s_part[i];
    }
    if (u > 0 && x >= lo && x < lo + u) {
      long long rel = x - lo;
      w.h = static_cast<int>(rel / walk.head_cost(w));
      rel -= w.h * walk.head_cost(w);
      const long long item = walk.start + static_cast<long long>(w.pages) * kCost2;
      w.blk = static_cast<int>(min(rel / item, static_cast<long long>(walk.last_blk(w))));
      rel -= w.blk * item;
      w.per = per;
      w.end = min(x + per, total);
      w.start = x - rel;
      w.pg0 = rel > walk.start ? static_cast<int>((rel - walk.start) / walk.page_cost(w, w.blk)) : 0;
      if (!walk.span(w)) w.b = -1;
      place = w;
    }
    __syncthreads();
    if (place.b >= 0 || before > x) break;
  }
  return place.b >= 0;
}

// On to the next block, head or row; false: the part ends.
static __device__ __noinline__ bool next_place(const Walk walk, Place& place, int* s_scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Place w = place;
  w.start += walk.item_cost(w, w.blk);
  w.pg0 = 0;
  bool more = w.start < w.end;
  if (more && w.blk++ == walk.last_blk(w)) {
    w.blk = 0;
    if (++w.h == walk.num_kv_heads) {
      w.h = 0;
      const int r1 = w.b + 1;
      int next = walk.num_rows;
      for (int r0 = r1; r0 < walk.num_rows && next == walk.num_rows; r0 += kThreads) {
        const unsigned has = __ballot_sync(0xffffffffu, walk.row(w, r0 + tid));
        if (lane == 0) s_scan[warp] = has ? r0 + warp * 32 + __ffs(has) - 1 : walk.num_rows;
        __syncthreads();
        for (int i = 0; i < kThreads / 32; ++i) next = min(next, s_scan[i]);
        __syncthreads();
      }
      more = walk.row(w, next);
    }
  }
  more = more && walk.span(w);
  __syncthreads();
  if (tid == 0) place = w;
  __syncthreads();
  return more;
}
}  // namespace pieces

template <int D, int G, int FMT, bool MOD>
__global__ void __launch_bounds__(pieces::kThreads, 1) gqa_pieces_kernel(const PartialArgs a, const pieces::Geo geo) {
  using namespace pieces;
  using Lt = Layout<D>;
  constexpr bool F16 = FMT != kBf16;
  constexpr int QT = kRows / G;   // tokens of one tile
  constexpr int QB = 2 * QT;      // tokens of a block
  constexpr int CH = D / 8;       // 16-byte pieces of a 16-bit row
  static_assert(G >= 1 && G <= 16 && (D == 64 || D == 128), "shape");
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_scan[kThreads / 32];
  __shared__ int s_row[3];  // row, first token, end token of this CTA's block
  __shared__ long long s_part[kThreads / 32];
  __shared__ Place s_place;
  __shared__ Item s_item;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform: roles branch without divergence
  const bool even = can_even(FMT) && geo.least > 0;  // equal parts of all rows; else a CTA a run (or a chunk of a stripe)
  const int P = a.P, z = blockIdx.z;
  int c = blockIdx.x;
  const int p0 = a.fused ? 0 : blockIdx.y / a.num_kv_heads;
  int h = blockIdx.y - p0 * a.num_kv_heads;
  const int t_real = __ldg(a.qo_indptr + a.num_rows);

  // ---- block z of padding tokens past the last row: 0 / -inf (chunk 0's CTAs)
  if (even) {
    const int64_t n = static_cast<int64_t>(max(0, a.num_tokens - t_real)) * a.num_kv_heads;
    for (int64_t x = blockIdx.x; x < n; x += gridDim.x)
      fused_zero_token(a, t_real + static_cast<int>(x / a.num_kv_heads), static_cast<int>(x % a.num_kv_heads), G, D);
  } else if (c == 0) {
    const int lo = t_real + z * QB, hi = min(lo + QB, a.num_tokens);
    for (int tok = lo; tok < hi; ++tok) {
      if (a.fused) {
        fused_zero_token(a, tok, h, G, D);
      } else {
        const int64_t orow0 = (static_cast<int64_t>(p0) * a.num_tokens + tok) * a.num_q_heads + h * G;
        for (int x = tid; x < G * D; x += blockDim.x) a.o_part[orow0 * D + x] = 0.f;
        if (tid < G) a.lse_part[lse_slot(a, p0, tok, h * G + tid)] = -INFINITY;
      }
    }
  }
  // ---- row block z: rows of >= 2 tokens in order, ceil(n / QB) blocks each (one-token rows are the
  // decode kernel's), found with a block-wide prefix sum over the rows
  int b = -1, s0 = 0, s1 = 0;
  const Walk walk = {a.qo_indptr, a.kv_len, a.num_rows, a.num_kv_heads, a.max_kv_len, a.page_size, geo.start, QT};
  if (even) {
    if (!first_place(walk, geo.least, s_place, s_part)) return;
  } else {
    if (tid == 0) s_row[0] = -1;
    int done_blocks = 0;
    for (int r0 = 0; r0 < a.num_rows; r0 += blockDim.x) {
      const int r = r0 + tid;
      int nb = 0, first = 0, n = 0;
      if (r < a.num_rows) {
        first = __ldg(a.qo_indptr + r);
        n = __ldg(a.qo_indptr + r + 1) - first;
        nb = n >= 2 ? (n + QB - 1) / QB : 0;
      }
      int incl = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      int before = done_blocks, total = done_blocks;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
      }
      const int lo = before + incl - nb;
      if (nb > 0 && z >= lo && z < lo + nb) {
        s_row[0] = r;
        s_row[1] = first + (z - lo) * QB;
        s_row[2] = min(first + n, first + (z - lo) * QB + QB);
      }
      done_blocks = total;
    }
    __syncthreads();
    b = s_row[0];
    if (b < 0) return;
    s0 = s_row[1];
    s1 = s_row[2];
  }
  bool tmem = false;
  // equal parts: every item of this CTA's part in turn
#pragma unroll 1
  for (;;) {
  // what an item derives from these is computed again for the next: kept across items it would cost the roles' loops
  // registers that they do not have
  const int tid = opaque(threadIdx.x), lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform: roles branch without divergence
  uint8_t* base = smem_raw + opaque(static_cast<int>((1024u - (tc05::smem_addr(smem_raw) & 1023u)) & 1023u));
  uint8_t* sK = base + Lt::OFF_K;
  uint8_t* sV = base + Lt::OFF_V;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + Lt::OFF_BAR);
  uint32_t* smask = reinterpret_cast<uint32_t*>(base + Lt::OFF_MASK);  // [slot][unit]: keys with data
  float* spos = reinterpret_cast<float*>(base + Lt::OFF_POS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + Lt::OFF_MISC);
  volatile int* s_abort = reinterpret_cast<volatile int*>(base + Lt::OFF_MISC + 4);
  int* spg = reinterpret_cast<int*>(base + Lt::OFF_PG);
  auto bar = [&](int i) { return tc05::smem_addr(&bars[i]); };
  if (even) {
    b = s_place.b;
    h = s_place.h;
    s0 = s_place.tok0 + s_place.blk * QB;
    s1 = s_place.tok0 + min(s_place.ntok, s_place.blk * QB + QB);
  }
  int L = __ldg(a.kv_len + b);
  if (L > a.max_kv_len) {
    if (c == 0 && tid == 0) report(a.dev_status, CPATTN_DEV_POS_PAST_TABLE);
    L = a.max_kv_len;
  }
  // ---- this CTA's keys: stripe slots [kb, kb + len) of partners p0 .. p0 + np - 1
  int nchunks, kb, len, np;
  if (even) {
    c = s_place.c;
    nchunks = s_place.nchunks;
    kb = s_place.pg0 * a.ps_l;
    len = max(0, static_cast<int>(min(static_cast<long long>(s_place.pg1 - s_place.pg0) * a.ps_l,
                                      static_cast<long long>(stripe_len(L, 0, P, a.interleave)) - kb)));
    np = P;
  } else if (a.fused) {
    nchunks = max(1, (L + geo.run - 1) / geo.run);
    // equal runs (16 rows of 2-256 tokens on up to 8192 E2M1 keys: 255 us; whole runs and a rest 264)
    const int n = (L + a.page_size - 1) / a.page_size;
    const int part = (n + nchunks - 1) / nchunks;
    kb = c * part * a.ps_l;
    len = max(0, min(part, n - c * part)) * a.ps_l;
    np = P;
  } else {
    const int n_p = stripe_len(L, p0, P, a.interleave);
    nchunks = n_p > 0 ? (n_p + a.chunk - 1) / a.chunk : 1;
    kb = c * a.chunk;
    len = max(0, min(n_p - kb, a.chunk));
    np = 1;
  }
  if (c >= nchunks) return;
  const int ntiles = (np * len + kTile - 1) / kTile;
  if (tid == 0) s_item = Item{c, nchunks, h, s0, s1, ntiles};
  __syncthreads();
  const int ntl = s1 - s0 > QT ? 2 : 1;          // query tiles with tokens
  const int my_t = warp >> 2;                    // softmax threads: tile, row, token, head
  const int my_r = (warp & 3) * 32 + lane;
  const int my_tok = s0 + my_t * QT + my_r / G;
  const int my_g = my_r % G;
  const bool my_ok = warp < kSoftWarps && my_tok < s1;

  float l = 0.f, m = -INFINITY;  // softmax rows: sum and running max (log2)
  bool alive = true;
  if (ntiles > 0) {
    // ---- page ids of the CTA's slots, checked once
    const int j0 = kb / a.ps_l;
    {
      const int j1 = (kb + len - 1) / a.ps_l;
      const int pb = __ldg(a.page_indptr + b);
      const int npages = __ldg(a.page_indptr + b + 1) - pb;
      for (int x = tid; x <= j1 - j0; x += blockDim.x) {
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
    if (tid == 0) {
      for (int i = 0; i < B_COUNT; ++i) {
        uint32_t cnt = 1;
        if (i < B_KFREE || (i >= B_VFULL && i < B_VFREE)) cnt = F16 ? kUnits : 32 * kUnits;
        if (i >= B_PFULL && i < B_PVDONE) cnt = 4;
        if (i == B_Q) cnt = 4 * ntl;
        if (tmem) tc05::mbar_inval(bar(i));  // every phase of the last item's is over
        tc05::mbar_init(bar(i), cnt);
      }
      *s_abort = 0;
      tc05::mbar_init_fence();
    }
    if (warp == 0 && !tmem) tc05::tmem_alloc(tc05::smem_addr(tmem_slot), Lt::TMEM_COLS);
    tmem = true;
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tbase = *tmem_slot;

    if (warp >= kLoadWarp) {
      // ================= copies =================
      const int li = warp - kLoadWarp;
      const bool is_k = li < kUnits;
      const int unit = li & (kUnits - 1);  // which 32 keys of a tile
      const uint8_t* pool = static_cast<const uint8_t*>(is_k ? a.pool_k : a.pool_v);
      const int nst = is_k ? kKStages : kVStages;
      uint8_t* ring = is_k ? sK : sV;
      const int b_full = is_k ? B_KFULL : B_VFULL, b_free = is_k ? B_KFREE : B_VFREE;
      // The lane's key of each tile: slot k of partner pp.  Tiles go from the
      // last to the first, a partner's keys from the nearest back: scores that
      // fall with the distance then meet their maximum at once (front to back
      // raised it, and rescaled O, at almost every tile of a steep head).
      const int x0 = unit * kUnit + lane;
      int pp = ((ntiles - 1) * kTile + x0) / len, k = kb + (ntiles - 1) * kTile + x0 - pp * len;
      int n_pp = stripe_len(L, p0 + min(pp, np - 1), P, a.interleave);
      // pool row of the lane's key of the next tile (-1: no key), its position counted from the row's end (exact in
      // float32 where it matters however long the row); advances the key
      auto next_row = [&](float& pos) -> int {
        int row = -1;
        if (pp < np && k < n_pp) {
          const int j = page_of_slot(a, k);
          const int pg = spg[j - j0];
          if (pg >= 0)
            row = static_cast<int>(((static_cast<int64_t>(p0 + pp) * a.num_pages + pg) * a.num_kv_heads + h) * a.ps_l +
                                   (k - j * a.ps_l));
          if (MOD && is_k) pos = static_cast<float>(stripe_pos(k, p0 + pp, P, a.interleave) - L);
        }
        k -= kTile;
        while (k < kb && pp > 0) {
          k += len;
          --pp;
          n_pp = stripe_len(L, p0 + min(pp, np - 1), P, a.interleave);
        }
        return row;
      };
      auto publish = [&](int i, int row, float pos) {  // written before the tile's copies (see kMaskSlots)
        const uint32_t vm = __ballot_sync(0xffffffffu, row >= 0);
        if (MOD) spos[(i % kMaskSlots) * kTile + x0] = pos;
        if (lane == 0) smask[(i % kMaskSlots) * kUnits + unit] = vm;
        __threadfence_block();
      };
      if constexpr (FMT == kBf16) {
        constexpr int RPI = 32 / CH;  // rows a warp instruction copies
        const int ro = lane / CH, cc = lane - (lane / CH) * CH;
        for (int i = 0; i < ntiles; ++i) {
          const int st = i % nst;
          if (i >= nst) {
            const bool ok = wait_phase(bar(b_free + st), ((i - nst) / nst) & 1, s_abort);
            if (!__all_sync(0xffffffffu, ok)) { alive = false; break; }
          }
          float pos = 0.f;
          const int myrow = next_row(pos);
          if (is_k) publish(i, myrow, pos);
          const uint32_t dst0 = tc05::smem_addr(ring) + st * Lt::TILE + (cc >> 3) * Lt::BLK;
#pragma unroll
          for (int u = 0; u < kUnit / RPI; ++u) {
            const int key = u * RPI + ro;
            const int row = __shfl_sync(0xffffffffu, myrow, key);
            const uint32_t dst = dst0 + tc05::sw128(unit * kUnit + key, cc & 7);
            if (row >= 0) ws_cp16(dst, pool + (static_cast<int64_t>(row) * D + cc * 8) * 2);
            else ws_cp16_zero(dst, pool);  // no key: zero row (finite scores, zero values)
          }
          ws_cp_arrive(bar(b_full + st));
        }
        cp_async_wait<0>();  // nothing lands after the CTA moves on
      } else {
        constexpr int CODES = FMT == kFp4 ? 32 : 16;  // values of a 16-byte piece
        constexpr int CHQ = D / CODES;                // pieces of a row
        constexpr int RPI = 32 / CHQ;                 // rows a warp instruction loads
        constexpr int NL = kUnit / RPI;               // pieces a lane takes of a tile
        const int ro = lane / CHQ, cq = lane - (lane / CHQ) * CHQ;
        struct Raw {  // a lane's pieces of one tile, as loaded
          uint4 codes[NL];
          uint32_t scl[NL], valid;
        };
        auto load = [&](Raw& r, int i) {
          float pos = 0.f;
          const int myrow = next_row(pos);
          if (is_k) publish(i, myrow, pos);
          r.valid = __ballot_sync(0xffffffffu, myrow >= 0);
#pragma unroll
          for (int u = 0; u < NL; ++u) {
            // keys without data load pool row 0 and are zeroed when they are converted: no branch, so every
            // load of the tile is in flight at once
            const int row = max(__shfl_sync(0xffffffffu, myrow, u * RPI + ro), 0);
            r.codes[u] = __ldg(reinterpret_cast<const uint4*>(pool + static_cast<int64_t>(row) * (D * 16 / CODES) + cq * 16));
            if constexpr (FMT == kFp4)
              r.scl[u] = __ldg(reinterpret_cast<const unsigned short*>(pool + a.scale_off +
                                                                       static_cast<int64_t>(row) * (D / 16) + cq * 2));
          }
        };
        // tile i out of `now`, the next one's loads into `next` first
        auto step = [&](Raw& now, Raw& next, int i) -> bool {
          const int st = i % nst;
          if (i + 1 < ntiles) load(next, i + 1);
          if (i >= nst) {
            const bool ok = wait_phase(bar(b_free + st), ((i - nst) / nst) & 1, s_abort);
            if (!__all_sync(0xffffffffu, ok)) return false;
          }
          uint8_t* dst0 = ring + st * Lt::TILE;
#pragma unroll
          for (int u = 0; u < NL; ++u) {
            const int key = unit * kUnit + u * RPI + ro;
            const uint32_t on = ((now.valid >> (u * RPI + ro)) & 1u) ? 0xffffffffu : 0u;
            const uint32_t w[4] = {now.codes[u].x & on, now.codes[u].y & on, now.codes[u].z & on, now.codes[u].w & on};
            // Pieces 8 apart lie in different column blocks at the same banks: the
            // lanes of the upper block take their pieces in another order, so the
            // eight lanes of a store phase hit all banks.
            const bool upper = cq >= CHQ / (D / 64);
            if constexpr (FMT == kFp4) {
              const uint32_t s2 = e4m3x2_to_f16x2(now.scl[u] & on);
#pragma unroll
              for (int x0 = 0; x0 < 4; ++x0) {  // 8 codes: one 16-byte piece of the row
                const int x = upper ? x0 ^ 2 : x0;
                const uint32_t wx = upper ? w[x0 ^ 2] : w[x0];
                const uint32_t sb = __byte_perm(s2, 0u, x < 2 ? 0x1010u : 0x3232u);
                const int cb = 4 * cq + x;
                *reinterpret_cast<uint4*>(dst0 + (cb >> 3) * Lt::BLK + tc05::sw128(key, cb & 7)) =
                    make_uint4(mul_f16x2(e2m1x2_to_f16x2<0>(wx), sb), mul_f16x2(e2m1x2_to_f16x2<1>(wx), sb),
                               mul_f16x2(e2m1x2_to_f16x2<2>(wx), sb), mul_f16x2(e2m1x2_to_f16x2<3>(wx), sb));
              }
            } else {
#pragma unroll
              for (int x0 = 0; x0 < 2; ++x0) {
                const int cb = 2 * cq + (upper ? x0 ^ 1 : x0);
                const uint32_t c0 = upper ? w[2 * (x0 ^ 1)] : w[2 * x0], c1 = upper ? w[2 * (x0 ^ 1) + 1] : w[2 * x0 + 1];
                *reinterpret_cast<uint4*>(dst0 + (cb >> 3) * Lt::BLK + tc05::sw128(key, cb & 7)) =
                    make_uint4(e4m3x2_to_f16x2(c0), e4m3x2_to_f16x2(c0 >> 16), e4m3x2_to_f16x2(c1),
                               e4m3x2_to_f16x2(c1 >> 16));
              }
            }
          }
          tc05::fence_smem_to_async();  // the tensor core reads what this lane wrote
          __syncwarp();
          if (lane == 0) ws_arrive(bar(b_full + st));
          return true;
        };
        Raw ra, rb;
        load(ra, 0);
        for (int i = 0; i < ntiles && alive; i += 2) {
          alive = step(ra, rb, i);
          if (alive && i + 1 < ntiles) alive = step(rb, ra, i + 1);
        }
      }
      if (!alive) *s_abort = 1;
    } else if (warp == kSWarp || warp == kPvWarp) {
      // ================= MMA issue =================
      // A whole warp walks the loop and one elected lane issues: control flow
      // stays uniform, so addresses and descriptors live in uniform registers
      // (a single-thread branch took about 20 cycles an instruction).
      const uint32_t bar0 = bar(0);
      bool issued = false;
      if (warp == kSWarp) {
        // S of each key tile for every query tile, as soon as P V of the tile before last has read its buffer
        constexpr uint32_t id_s = F16 ? tc05::idesc_f16(128, kTile, false, false) : tc05::idesc_bf16(128, kTile, false, false);
        const uint64_t dq = tc05::desc_k128(tc05::smem_addr(base));
        const uint64_t dk0 = tc05::desc_k128(tc05::smem_addr(sK));
        alive = wait_phase(bar0 + 8 * B_Q, 0, s_abort);
        uint32_t st = 0, ph = 0;  // ring stage and phase
        for (int j = 0; j < ntiles && alive; ++j) {
          alive = wait_phase(bar0 + 8 * (B_KFULL + st), ph, s_abort);
          if constexpr (!F16) tc05::fence_smem_to_async();  // cp.async wrote through the generic proxy
          const uint64_t dk = tc05::desc_add(dk0, st * Lt::TILE);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t < ntl && alive) {
              if (j > 1) alive = wait_phase(bar0 + 8 * (B_PVDONE + 2 * t + (j & 1)), ((j >> 1) - 1) & 1, s_abort);
              tc05::fence_after_sync();
              if (alive && tc05::elect_one()) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                  tc05::mma_ss(tbase + t * Lt::TILE_COLS + Lt::S_COLS * (j & 1),
                               tc05::desc_add(dq, t * Lt::QTILE + (s >> 2) * Lt::QBLK + (s & 3) * 32),
                               tc05::desc_add(dk, (s >> 2) * Lt::BLK + (s & 3) * 32), id_s, s > 0);
                tc05::commit(bar0 + 8 * (B_SDONE + 2 * t + (j & 1)));
                if (t == ntl - 1) tc05::commit(bar0 + 8 * (B_KFREE + st));
              }
              __syncwarp();
              issued = true;
            }
          }
          if (++st == kKStages) st = 0, ph ^= 1;
        }
        for (int j = max(0, ntiles - kKStages); j < ntiles && alive; ++j)
          alive = wait_phase(bar0 + 8 * (B_KFREE + j % kKStages), (j / kKStages) & 1, s_abort);
      } else {
        constexpr uint32_t id_o = F16 ? tc05::idesc_f16(128, D, false, true) : tc05::idesc_bf16(128, D, false, true);
        const uint64_t dv0 = tc05::desc_mn128(tc05::smem_addr(sV), Lt::BLK);
        uint32_t st = 0, ph = 0;
        for (int j = 0; j < ntiles && alive; ++j) {
          alive = wait_phase(bar0 + 8 * (B_VFULL + st), ph, s_abort);
          if constexpr (!F16) tc05::fence_smem_to_async();
          const uint64_t dv = tc05::desc_add(dv0, st * Lt::TILE);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t < ntl && alive) {
              alive = wait_phase(bar0 + 8 * (B_PFULL + 2 * t + (j & 1)), (j >> 1) & 1, s_abort);
              tc05::fence_after_sync();
              const uint32_t tt = tbase + t * Lt::TILE_COLS;
              if (alive && tc05::elect_one()) {
#pragma unroll
                for (int s = 0; s < kTile / 16; ++s)
                  tc05::mma_ts(tt + Lt::O_COL, tt + Lt::S_COLS * (j & 1) + 8 * s, tc05::desc_add(dv, s * 16 * 128),
                               id_o, j > 0 || s > 0);
                tc05::commit(bar0 + 8 * (B_PVDONE + 2 * t + (j & 1)));
                if (t == ntl - 1) tc05::commit(bar0 + 8 * (B_VFREE + st));
              }
              __syncwarp();
              issued = true;
            }
          }
          if (++st == kVStages) st = 0, ph ^= 1;
        }
        for (int j = max(0, ntiles - kVStages); j < ntiles && alive; ++j)
          alive = wait_phase(bar0 + 8 * (B_VFREE + j % kVStages), (j / kVStages) & 1, s_abort);
      }
      if (!alive) {
        *s_abort = 1;
        if (issued) {  // no MMA may still run when the tensor memory is released
          const uint32_t fin = bar0 + 8 * (B_FIN + warp - kSWarp);
          if (tc05::elect_one()) tc05::commit(fin);
          __syncwarp();
          tc05::mbar_wait(fin, 0, 1u << 20);
        }
      }
    } else if (warp < kSoftWarps && my_t < ntl) {
      // ================= softmax rows =================
      const uint32_t my_lane = tc05::taddr(tbase, (warp & 3) * 32, my_t * Lt::TILE_COLS);
      const float kscale = a.scale * (F16 ? a.k_descale : 1.f);
      const float sl = MOD ? 1.f : kscale * kLog2e;
      ScoreMod smod;
      float slope2 = 0.f, qpos = 0.f;
      if constexpr (MOD) {
        smod = score_mod_of(a.softcap, kscale);
        if (a.slopes != nullptr && my_ok) {
          slope2 = __ldg(a.slopes + h * G + my_g) * kLog2e;
          qpos = static_cast<float>(query_pos(a, b, my_tok, __ldg(a.qo_indptr + b)) - L);
        }
      }
      {  // this thread's query row, in the MMA layout (and type)
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) +
                                                          (static_cast<int64_t>(my_tok) * a.num_q_heads + h * G + my_g) * D * 2);
        uint8_t* dst = base + my_t * Lt::QTILE;
#pragma unroll
        for (int c0 = 0; c0 < CH; c0 += 8) {
          uint4 w[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) w[x] = my_ok ? __ldg(src + c0 + x) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            if constexpr (F16)
              w[x] = make_uint4(bf16x2_to_f16x2(w[x].x), bf16x2_to_f16x2(w[x].y), bf16x2_to_f16x2(w[x].z),
                                bf16x2_to_f16x2(w[x].w));
            *reinterpret_cast<uint4*>(dst + ((c0 + x) >> 3) * Lt::QBLK + tc05::sw128(my_r, x)) = w[x];
          }
        }
        tc05::fence_smem_to_async();
        __syncwarp();
        if (lane == 0) ws_arrive(bar(B_Q));
      }
      for (int i = 0; i < ntiles; ++i) {
        const int bb = i & 1;
        bool ok = wait_phase(bar(B_SDONE + 2 * my_t + bb), (i >> 1) & 1, s_abort);
        if (!__all_sync(0xffffffffu, ok)) { alive = false; break; }
        tc05::fence_after_sync();
        const uint32_t mlo = smask[(i % kMaskSlots) * kUnits], mhi = smask[(i % kMaskSlots) * kUnits + 1];
        const uint32_t s_lane = my_lane + Lt::S_COLS * bb;
        float sv[kTile];
        {
          float v0[16], v1[16], v2[16], v3[16];
          tc05::ld_x16(s_lane, v0);
          tc05::ld_x16(s_lane + 16, v1);
          tc05::ld_x16(s_lane + 32, v2);
          tc05::ld_x16(s_lane + 48, v3);
          tc05::ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            sv[e] = v0[e];
            sv[16 + e] = v1[e];
            sv[32 + e] = v2[e];
            sv[48 + e] = v3[e];
          }
        }
        if constexpr (MOD) {
          const float4* kp = reinterpret_cast<const float4*>(spos + (i % kMaskSlots) * kTile);
          if (a.slopes == nullptr) {
            if (smod.kind == kCapPlain) modify<kCapPlain, false>(smod, sv, 0.f, 0.f, kp);
            else modify<kCapSeries, false>(smod, sv, 0.f, 0.f, kp);
          } else if (smod.kind == kCapNone) {
            modify<kCapNone, true>(smod, sv, slope2, qpos, kp);
          } else if (smod.kind == kCapPlain) {
            modify<kCapPlain, true>(smod, sv, slope2, qpos, kp);
          } else {
            modify<kCapSeries, true>(smod, sv, slope2, qpos, kp);
          }
        }
        // keys without data: -inf (probability 0)
        if ((mlo & mhi) != 0xffffffffu) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            sv[e] = ((mlo >> e) & 1u) ? sv[e] : -INFINITY;
            sv[32 + e] = ((mhi >> e) & 1u) ? sv[32 + e] : -INFINITY;
          }
        }
        float mx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          mx[e] = fmaxf(sv[e], sv[8 + e]);
#pragma unroll
          for (int w = 2; w < 8; w += 2) mx[e] = max3(mx[e], sv[8 * w + e], sv[8 * w + 8 + e]);
        }
        const float bm = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sl;
        const bool up = bm > m + 8.f;
        if (__any_sync(0xffffffffu, up) && i > 0) {
          // rescale O rows whose max rose; P V of the previous tile must be done (S of this tile came after
          // P V of the tile before it, so the wait cannot see an older phase)
          ok = wait_phase(bar(B_PVDONE + 2 * my_t + ((i - 1) & 1)), ((i - 1) >> 1) & 1, s_abort);
          if (!__all_sync(0xffffffffu, ok)) { alive = false; break; }
          tc05::fence_after_sync();
          const float alpha = up ? exp2f(m - bm) : 1.f;
#pragma unroll
          for (int col = 0; col < D; col += 16) {
            float v[16];
            tc05::ld_x16(my_lane + Lt::O_COL + col, v);
            tc05::ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= alpha;
            tc05::st_x16(my_lane + Lt::O_COL + col, v);
          }
          tc05::st_wait();
          l *= alpha;
        }
        if (up) m = bm;
        // one FMA and one ex2 a key (-inf gives 0; while every key so far is
        // masked m is -inf and every p is 0)
        const float nm = m == -INFINITY ? 0.f : -m;
        const uint64_t sl2 = pair2(sl, sl), nm2 = pair2(nm, nm);
        uint64_t ls[2] = {0ull, 0ull};  // pairs of partial sums
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float pa, pb;
            unpair2(fma2(pair2(sv[32 * hh + 2 * e], sv[32 * hh + 2 * e + 1]), sl2, nm2), pa, pb);
            pa = ex2_approx(pa);
            pb = ex2_approx(pb);
            ls[e & 1] = add2(ls[e & 1], pair2(pa, pb));
            pk[e] = pack16<F16>(pa, pb);
          }
          tc05::st_x16_u32(s_lane + 16 * hh, pk);
        }
        {
          float s0, s1;
          unpair2(add2(ls[0], ls[1]), s0, s1);
          l += s0 + s1;
        }
        tc05::st_wait();
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) ws_arrive(bar(B_PFULL + 2 * my_t + bb));
      }
      if (alive) {
        bool ok = true;
        for (int i = max(0, ntiles - 2); i < ntiles; ++i)
          ok = ok && wait_phase(bar(B_PVDONE + 2 * my_t + (i & 1)), (i >> 1) & 1, s_abort);
        alive = __all_sync(0xffffffffu, ok);
      }
      if (!alive) *s_abort = 1;
    }
  }

  // ---- softmax rows: output, or a normalised piece with its LSE.  (What the item's loops need not know is read, or
  // computed, again.)
  {
  const Item it = s_item;
  const int c = it.c, nchunks = it.nchunks, h = it.h, s0 = it.s0, s1 = it.s1, ntiles = it.ntiles;
  const int tid = opaque(threadIdx.x), lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t tbase = ntiles > 0 ? *tmem_slot : 0u;
  const bool single = nchunks == 1;
  const int ntl = s1 - s0 > QT ? 2 : 1;
  const int my_t = warp >> 2;
  const int my_r = (warp & 3) * 32 + lane;
  const int my_tok = s0 + my_t * QT + my_r / G;
  const int my_g = my_r % G;
  const bool my_ok = warp < kSoftWarps && my_tok < s1;
  if (warp < kSoftWarps && my_t < ntl && alive) {
    tc05::fence_after_sync();
    const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    float w = l > 0.f ? (F16 ? a.v_descale : 1.f) / l : 0.f, we = 0.f;  // weights of this piece, of the extra partial
    float lse_all = lse;
    const int64_t hq = static_cast<int64_t>(my_tok) * a.num_q_heads + h * G + my_g;
    const bool final = a.fused && single;
    if (final && a.extra_lse != nullptr && my_ok) {
      const float le = __ldg(a.extra_lse + hq);
      const float mm = fmaxf(lse, le);
      if (mm != -INFINITY) {
        const float e0 = expf(lse - mm), e1 = expf(le - mm);
        w *= e0 / (e0 + e1);
        we = e1 / (e0 + e1);
        lse_all = mm + logf(e0 + e1);
      }
    }
    float* dst = nullptr;
    float* ldst = nullptr;
    if (final) {
      ldst = a.lse_out != nullptr ? a.lse_out + hq : nullptr;
    } else if (a.fused) {
      const int64_t wrow = ((static_cast<int64_t>(my_tok) * a.num_kv_heads + h) * geo.max_runs + c) * G + my_g;
      dst = geo.ws_o + wrow * D;
      ldst = geo.ws_lse + wrow;
      if (my_ok && my_g == 0 && c == nchunks - 1) a.ws_pair[static_cast<int64_t>(my_tok) * a.num_kv_heads + h] = nchunks;
    } else if (single) {
      dst = a.o_part + ((static_cast<int64_t>(p0) * a.num_tokens) * a.num_q_heads + hq) * D;
      ldst = a.lse_part + lse_slot(a, p0, my_tok, h * G + my_g);
    } else {
      const int64_t slot = (static_cast<int64_t>(my_tok) * P + p0) * a.num_kv_heads + h;
      const int64_t wrow = (slot * a.max_chunks + c) * G + my_g;
      dst = a.ws_o + wrow * D;
      ldst = a.ws_lse + wrow;
    }
    // Rows leave through the tile's query area (its last S is done): a lane lays
    // out its row, or half of a float32 one, and sends it with one bulk copy.
    // Storing rows from the lanes took 12k cycles a CTA: 32 rows an instruction.
    const uint32_t o_lane = tc05::taddr(tbase, (warp & 3) * 32, my_t * Lt::TILE_COLS) + Lt::O_COL;
    constexpr int RB = Lt::QTILE / kRows;  // bytes of a staged row: D values of 16 bits or D / 2 of 32
    uint8_t* stage = base + my_t * Lt::QTILE + my_r * RB;
    const bool half_rows = !(final && a.out_bf16);
    uint8_t* gdst = final ? static_cast<uint8_t*>(a.out) + hq * D * (a.out_bf16 ? 2 : 4) : reinterpret_cast<uint8_t*>(dst);
#pragma unroll 1
    for (int col = 0; col < D; col += 32) {
      float v[32];
      __syncwarp();
      if (ntiles > 0) {
        float v0[16], v1[16];
        tc05::ld_x16(o_lane + col, v0);  // warp-collective: every lane loads
        tc05::ld_x16(o_lane + col + 16, v1);
        tc05::ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = v0[e] * w, v[16 + e] = v1[e] * w;
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0.f;
      }
      if (!my_ok) continue;
      if (we != 0.f) {  // an empty extra partial's row is never read
        float4 x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __ldg(reinterpret_cast<const float4*>(a.extra_o + hq * D + col) + e);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[4 * e] = fmaf(we, x[e].x, v[4 * e]);
          v[4 * e + 1] = fmaf(we, x[e].y, v[4 * e + 1]);
          v[4 * e + 2] = fmaf(we, x[e].z, v[4 * e + 2]);
          v[4 * e + 3] = fmaf(we, x[e].w, v[4 * e + 3]);
        }
      }
      if (half_rows) {
        if (col == D / 2) tc05::bulk_wait_read();  // the first half has left
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4*>(stage + (col & (D / 2 - 1)) * 4 + e * 16) =
              make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        if (((col + 32) & (D / 2 - 1)) == 0) {
          tc05::fence_smem_to_async();
          bulk_s2g(gdst + (col + 32 - D / 2) * 4, tc05::smem_addr(stage), RB);
          tc05::bulk_commit();
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(stage + col * 2 + e * 16) =
              make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                         pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
        if (col + 32 == D) {
          tc05::fence_smem_to_async();
          bulk_s2g(gdst, tc05::smem_addr(stage), RB);
          tc05::bulk_commit();
        }
      }
    }
    tc05::bulk_wait_all();
    if (my_ok && ldst != nullptr) *ldst = lse_all;
  }
  tc05::fence_before_sync();
  __syncthreads();
  const bool failed = ntiles > 0 && *s_abort != 0;
  if (failed && tid == 0) report(a.dev_status, CPATTN_DEV_TC_TIMEOUT);
  if (even && !failed && next_place(walk, s_place, s_scan)) continue;
  if (tmem && warp == 0) tc05::tmem_dealloc(tbase, Lt::TMEM_COLS);
  if (failed || single || a.fused) return;  // fused rows of several pieces: gqa_pieces_merge_kernel
  // ---- per-partner calls: the stripe's last CTA merges its chunks
  const int64_t slot0 = (static_cast<int64_t>(s0) * P + p0) * a.num_kv_heads + h;
  if (!take_ticket(a.ws_cnt + slot0, nchunks)) return;
  merge_chunks<kMergeUnroll>(a, p0, h, s0, s1 - s0, slot0, static_cast<int64_t>(P) * a.num_kv_heads, nchunks, G, D,
                             reinterpret_cast<float*>(base), Lt::SCRATCH);
  if (tid == 0) a.ws_cnt[slot0] = 0;
  return;
  }
  }
}

// Fused calls: the exact merge of an item's pieces and the extra partial, a
// block eight heads of a token and a warp two of them.  Its own kernel, because a
// block's last CTA alone took 34 us for the 256 rows of its merge (a row of E
// pieces is E + 1 short reads, which one SM cannot keep enough of in flight).
// What it spends is the chain of dependent small reads (number of pieces, LSEs,
// values), so blocks are many and light: about 25 us for 2064 tokens of 32
// heads; four heads a warp at 128 registers took 35.
template <int D>
__global__ void __launch_bounds__(32 * pieces::kMergeWarps, 8)
    gqa_pieces_merge_kernel(const PartialArgs a, const pieces::Geo geo, int G) {
  pdl_wait();
  using pieces::kMergeWarps;
  constexpr int NH = 2;            // heads a warp merges together
  constexpr int LN = D / 4;        // lanes a row takes
  constexpr int PARTS = 32 / LN;   // pieces read at once
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x;
  const int part = lane / LN, c4 = lane - part * LN;
  for (int h0 = (blockIdx.y * kMergeWarps + warp) * NH; h0 < a.num_q_heads; h0 += gridDim.y * kMergeWarps * NH) {
    int E[NH], most = 0;      // pieces (0: the item's only CTA wrote its output, or the token's row has no other
                              // token: its ticket here is 0 again)
    int64_t w0[NH], row[NH];  // piece e of head i: workspace row w0 + e G
    float le[NH], mx[NH], sum[NH];
    float4 acc[NH], vx[NH];
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const int hq = min(h0 + i, a.num_q_heads - 1);  // past the last head: its work again, not written
      row[i] = static_cast<int64_t>(t) * a.num_q_heads + hq;
      const int64_t item = static_cast<int64_t>(t) * a.num_kv_heads + hq / G;
      E[i] = __ldg(a.ws_pair + item);
      most = max(most, E[i]);
      w0[i] = item * geo.max_runs * G + hq % G;
      le[i] = a.extra_lse != nullptr ? __ldg(a.extra_lse + row[i]) : -INFINITY;
      vx[i] = acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      sum[i] = 0.f;
    }
    if (most == 0) continue;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      mx[i] = le[i];
      for (int e = lane; e < E[i]; e += 32) mx[i] = fmaxf(mx[i], __ldg(geo.ws_lse + w0[i] + static_cast<int64_t>(e) * G));
      if (le[i] != -INFINITY) vx[i] = __ldg(reinterpret_cast<const float4*>(a.extra_o + row[i] * D) + c4);
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
      if (mx[i] == -INFINITY) mx[i] = 0.f;  // no keys anywhere: every weight 0
    }
    for (int e0 = 0; e0 < most; e0 += 32) {
      float we[NH];
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        we[i] = e0 + lane < E[i] ? expf(__ldg(geo.ws_lse + w0[i] + static_cast<int64_t>(e0 + lane) * G) - mx[i]) : 0.f;
        sum[i] += we[i];
      }
      const int n = min(32, most - e0);
#pragma unroll 2
      for (int eb = 0; eb < n; eb += PARTS) {
        const int e = eb + part;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          const float x = __shfl_sync(0xffffffffu, we[i], e & 31);
          if (e < n && x != 0.f) {  // an empty piece's row is never read
            const float4 v =
                __ldg(reinterpret_cast<const float4*>(geo.ws_o + (w0[i] + static_cast<int64_t>(e0 + e) * G) * D) + c4);
            acc[i].x = fmaf(x, v.x, acc[i].x);
            acc[i].y = fmaf(x, v.y, acc[i].y);
            acc[i].z = fmaf(x, v.z, acc[i].z);
            acc[i].w = fmaf(x, v.w, acc[i].w);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
      if constexpr (PARTS == 2) {
        acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, 16);
        acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, 16);
        acc[i].z += __shfl_xor_sync(0xffffffffu, acc[i].z, 16);
        acc[i].w += __shfl_xor_sync(0xffffffffu, acc[i].w, 16);
      }
      const float wx = le[i] == -INFINITY ? 0.f : expf(le[i] - mx[i]);
      acc[i].x = fmaf(wx, vx[i].x, acc[i].x);
      acc[i].y = fmaf(wx, vx[i].y, acc[i].y);
      acc[i].z = fmaf(wx, vx[i].z, acc[i].z);
      acc[i].w = fmaf(wx, vx[i].w, acc[i].w);
      sum[i] += wx;
      if (h0 + i >= a.num_q_heads || E[i] == 0) continue;
      const float inv = sum[i] > 0.f ? 1.f / sum[i] : 0.f;
      if (part == 0) {
        const int64_t oi = row[i] * D + c4 * 4;
        if (a.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + oi) =
              make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + oi) =
              make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
      }
      if (lane == 0 && a.lse_out != nullptr) a.lse_out[row[i]] = sum[i] > 0.f ? mx[i] + logf(sum[i]) : -INFINITY;
    }
  }
}

namespace pieces {
template <int D, int G, int FMT, bool MOD>
int launch_t(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  constexpr int QB = 2 * kRows / G;
  Geo geo = {};
  int page_slots;
  if (a.fused) {
    // The pieces lie where the per-partner kernels keep theirs (this launch
    // starts when theirs are done), with room for P * max_chunks a token and
    // head; or where the decode kernel over E2M1 pools keeps its max_runs.
    int64_t room = static_cast<int64_t>(a.P) * a.max_chunks;
    geo.ws_o = a.max_chunks > 1 ? a.ws_o : a.o_part;
    geo.ws_lse = a.max_chunks > 1 ? a.ws_lse : a.lse_part;
    if (FMT == kFp4 && a.max_runs > room) {
      room = a.max_runs;
      geo.ws_o = a.ws_run_o;
      geo.ws_lse = a.ws_run_lse;
    }
    const int64_t blocks = static_cast<int64_t>(a.num_kv_heads) * ((a.num_tokens + QB - 1) / QB);
    auto runs = [&](int positions) {
      geo.run = (positions + a.page_size - 1) / a.page_size * a.page_size;
      geo.max_runs = a.max_kv_len > 0 ? (a.max_kv_len + geo.run - 1) / geo.run : 1;
    };
    // Longer runs where there are CTAs enough all the same: half the pieces to
    // merge (16 rows of 2-256 tokens on up to 8192 E2M1 keys: 239 us, runs of
    // 2048 250, of 8192 272).
    runs(kRun);
    if (geo.max_runs * blocks > 4 * kSms) {
      runs(2 * kRun);
    } else if (geo.max_runs * blocks < kSms) {  // few: shorter ones reach more SMs
      const int64_t fit = (a.max_kv_len + room - 1) / room, want = (a.max_kv_len * blocks + kSms - 1) / kSms;
      const int64_t least = fit > want ? fit : want;
      runs(least < 256 ? 256 : (least < kRun ? static_cast<int>(least) : kRun));
    }
    page_slots = geo.run / a.page_size + 1;
    // A CTA a run where that is about one round of CTAs.  Else all rows' pages
    // in equal parts, one a CTA, as long as a part's page ids fit: whole items
    // need no merge, and every SM ends at the same time (16 rows of 2-256
    // tokens on up to 8192 bf16 keys, both modifications: 290 us for 301).
    const int64_t pages = (static_cast<int64_t>(a.max_kv_len) + a.page_size - 1) / a.page_size;
    if (can_even(FMT) && geo.max_runs * blocks > kSms && room > 1 &&
        Layout<D>::smem_bytes(0) + 4 * (pages + 1) <= 227 * 1024) {
      geo.least = (pages * kCost2 + room - 2) / (room - 1);
      geo.start = (kStart * kCost2 + a.page_size - 1) / a.page_size;
      page_slots = static_cast<int>(pages) + 1;
    }
    if (geo.max_runs > room) return CPATTN_ERR_UNSUPPORTED_SHAPE;
    if (geo.least > 0) geo.max_runs = static_cast<int>(room);
  } else {
    geo.max_runs = a.max_chunks;
    page_slots = a.chunk / a.ps_l + 2;
  }
  const size_t smem = Layout<D>::smem_bytes(page_slots);
  if (smem > 227 * 1024) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  // the copy warps exchange pool row indices as 32-bit values
  if (static_cast<int64_t>(a.P) * a.num_pages * a.num_kv_heads * a.ps_l >= (int64_t{1} << 31))
    return CPATTN_ERR_UNSUPPORTED_SHAPE;
  auto kern = gqa_pieces_kernel<D, G, FMT, MOD>;
  static std::atomic<int> smem_set[64];
  *err = ensure_smem(kern, smem, smem_set);
  if (*err != cudaSuccess) return CPATTN_ERR_CUDA;
  // row blocks: at most one partial block a row beyond T / QB full ones (the
  // first T / QB of them also cover the blocks of padding tokens)
  const int qblocks = (a.num_tokens + QB - 1) / QB;
  const dim3 grid = geo.least > 0 ? dim3(kSms) : dim3(geo.max_runs, (a.fused ? 1 : a.P) * a.num_kv_heads, a.num_rows + qblocks);
  kern<<<grid, kThreads, smem, s>>>(a, geo);
  *err = cudaGetLastError();
  if (*err == cudaSuccess && a.fused && geo.max_runs > 1) {
    *err = launch_pdl(gqa_pieces_merge_kernel<D>, dim3(a.num_tokens, (a.num_q_heads + 2 * kMergeWarps - 1) / (2 * kMergeWarps)), dim3(32 * kMergeWarps), 0, s, a, geo, G);
  }
  return *err == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

template <int D, int FMT, bool MOD>
int dispatch_g(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch_t<D, 1, FMT, MOD>(a, s, err);
    case 2: return launch_t<D, 2, FMT, MOD>(a, s, err);
    case 4: return launch_t<D, 4, FMT, MOD>(a, s, err);
    case 8: return launch_t<D, 8, FMT, MOD>(a, s, err);
    case 16: return launch_t<D, 16, FMT, MOD>(a, s, err);
    default: return CPATTN_ERR_UNSUPPORTED_SHAPE;
  }
}

template <int FMT, bool MOD>
int dispatch(const PartialArgs& a, cudaStream_t s, cudaError_t* err) {
  if (a.head_dim == 128) return dispatch_g<128, FMT, MOD>(a, s, err);
  if (a.head_dim == 64) return dispatch_g<64, FMT, MOD>(a, s, err);
  return CPATTN_ERR_UNSUPPORTED_SHAPE;
}
}  // namespace pieces

}  // namespace cpattn
