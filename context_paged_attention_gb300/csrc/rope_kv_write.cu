// cp_rope_kv_write: rotate a step's queries and new keys by their positions
// and write the new K/V into the P-way striped paged pool, in one launch.
//
// A pair (u, v) of a row at position n turns by the angle whose cosine c and
// sine s the caller's table holds for n:  u' = u c - v s,  v' = v c + u s.
// Pairs are (i, i + r / 2) ("halves") or (2 i, 2 i + 1) ("pairs") of the r
// rotated values; the other values pass through.  The products and the sum are
// taken in float32, each rounded (no fused multiply-add: a row comes out with
// the same bits however the compiler schedules it), and the result is rounded
// once to each output: the layer's type for q_out and k_out, and for the pool
// its own type -- E4M3 and E2M1 codes come from the float32 values, not from
// the rounded k_out.  Values are not rotated; they reach the pool as
// cp_kv_write writes them.
#include "kv_quant.cuh"

namespace cpattn {

namespace {
constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = 256;
constexpr int kRopeManyTokens = 608;  // a block a token fills the SMs four times: rows share a thread from here on

template <typename T>
__device__ __forceinline__ float load_f(const T* p);
template <>
__device__ __forceinline__ float load_f(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
}

// NB float32 values -> NB values of type T (nearest even), 16 bytes a store.
template <typename T, int NB>
__device__ __forceinline__ void store_row_piece(T* dst, const float (&x)[NB]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < NB; i += 4)
      reinterpret_cast<float4*>(dst)[i / 4] = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < NB; i += 8) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[i + 2 * j], x[i + 2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      reinterpret_cast<uint4*>(dst)[i / 8] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Values [e0, e0 + NB) of a pool row of d values, in the pool's type.
template <typename T, int QUANT, int NB>
__device__ __forceinline__ void store_pool_piece(void* pool, int64_t prow, int d, int e0, const float (&x)[NB],
                                                 float descale, int64_t scale_off) {
  uint8_t* base = static_cast<uint8_t*>(pool);
  if constexpr (QUANT == kQuantNone) {
    store_row_piece<T, NB>(reinterpret_cast<T*>(pool) + prow * d + e0, x);
  } else if constexpr (QUANT == kQuantE4m3) {
    static_assert(NB == 8, "8 codes a store");
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4] |= e4m3_rn_satfinite(__fdiv_rn(x[i], descale)) << (8 * (i & 3));
    *reinterpret_cast<uint2*>(base + prow * d + e0) = make_uint2(w[0], w[1]);
  } else {
    static_assert(NB == 16, "one scale block a store");
    uint2 codes;
    uint32_t scale;
    fp4_encode_block(x, descale, codes, scale);
    *reinterpret_cast<uint2*>(base + (prow * d + e0) / 2) = codes;
    base[scale_off + (prow * d + e0) / 16] = static_cast<uint8_t>(scale);
  }
}
}  // namespace

// A warp takes one row (a query, key or value head of one token): the row goes
// through shared memory as float32, so any rotated width and offset works and
// q_out / k_out may be the inputs themselves.
template <typename T, int QUANT>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_rows_kernel(const RopeArgs a) {
  constexpr int NB = QUANT == kQuantFp4 ? 16 : (sizeof(T) == 4 ? 4 : 8);  // values a lane writes at once
  extern __shared__ float srow[];
  pdl_trigger();
  pdl_wait();
  const WriteArgs& w = a.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nq = a.q != nullptr ? a.num_q_heads : 0;
  const int nv = w.pool_v != nullptr ? w.num_kv_heads : 0;
  const int per_token = nq + w.num_kv_heads + nv;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  const int t = static_cast<int>(item / per_token);
  if (t >= w.num_tokens) return;
  int r = static_cast<int>(item - static_cast<int64_t>(t) * per_token);
  const int b = row_of_token(w.qo_indptr, w.num_rows, t);
  if (b < 0) return;
  const int pos = __ldg(w.positions + t);
  if (pos < 0) return;  // padding token
  if (pos >= a.table_len) {
    if (r == 0 && lane == 0) report(w.dev_status, CPATTN_DEV_POS_PAST_ROPE);
    return;
  }
  // kind of row: 0 query, 1 key, 2 value
  const int kind = r < nq ? 0 : (r < nq + w.num_kv_heads ? 1 : 2);
  r -= kind == 0 ? 0 : (kind == 1 ? nq : nq + w.num_kv_heads);
  const int d = kind == 2 ? a.head_dim_v : a.head_dim;
  const int64_t srow_idx = static_cast<int64_t>(t) * (kind == 0 ? a.num_q_heads : w.num_kv_heads) + r;
  const T* src = static_cast<const T*>(kind == 0 ? a.q : (kind == 1 ? w.k_new : w.v_new)) + srow_idx * d;
  float* x = srow + static_cast<size_t>(warp) * a.head_dim;
  for (int e = lane; e < d; e += 32) x[e] = load_f(src + e);
  __syncwarp();
  int64_t prow = -1;
  if (kind != 0) {
    const int64_t row0 = pool_row0(w, b, pos, kind == 1 && r == 0 && lane == 0);
    if (row0 >= 0) prow = row0 + static_cast<int64_t>(r) * (w.page_size / w.P);
  }
  const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim;
  const int half = a.rot_dim / 2;
  T* out = static_cast<T*>(kind == 0 ? a.q_out : (kind == 1 ? a.k_out : nullptr));
  for (int e0 = lane * NB; e0 < d; e0 += 32 * NB) {
    float y[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int e = e0 + i, j = e - a.rot_begin;
      y[i] = x[e];
      if (kind != 2 && j >= 0 && j < a.rot_dim) {
        const bool second = a.pairs ? (j & 1) : j >= half;
        const int f = a.pairs ? j >> 1 : (second ? j - half : j);
        const int mate = a.pairs ? (second ? e - 1 : e + 1) : (second ? e - half : e + half);
        const float c = __ldg(cs + f), s = __ldg(cs + half + f);
        const float xs = __fmul_rn(x[mate], s);
        y[i] = __fadd_rn(__fmul_rn(y[i], c), second ? xs : -xs);
      }
    }
    if (out != nullptr) store_row_piece<T, NB>(out + srow_idx * d + e0, y);
    if (prow >= 0) {
      if (kind == 1) store_pool_piece<T, QUANT, NB>(w.pool_k, prow, d, e0, y, w.k_descale, w.scale_off_k);
      else store_pool_piece<T, QUANT, NB>(w.pool_v, prow, d, e0, y, w.v_descale, w.scale_off_v);
    }
  }
}

// The common shapes (rotated width and start, and head width, multiples of 16;
// for rotated halves over E2M1 pools the width a multiple of 32): a thread
// takes 16 values of a row as two pieces of 8 -- a rotated half's piece and its
// mate's, two neighbouring pieces otherwise -- so every pair turns inside the
// thread, q_out / k_out may be the inputs, and loads and stores are whole
// 16-byte pieces.  It takes the same unit of up to kRows rows (heads) of its
// token: one position, one set of cosines and sines and one page lookup serve
// them, and all their loads are in flight together.
template <typename T>
struct Piece16 {  // 16 values as loaded: two pieces of 8
  static constexpr int N = sizeof(T) == 4 ? 2 : 1;
  uint4 a[N], b[N];
  __device__ __forceinline__ void load(const T* pa, const T* pb) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = __ldg(reinterpret_cast<const uint4*>(pa) + i);
      b[i] = __ldg(reinterpret_cast<const uint4*>(pb) + i);
    }
  }
  __device__ __forceinline__ void widen(float* x) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      Chunk16<T>::widen(a[i], x + i * Chunk16<T>::N);
      Chunk16<T>::widen(b[i], x + 8 + i * Chunk16<T>::N);
    }
  }
};

// Four float32 values -> four E4M3 codes (cvt's saturation, ties and NaN are
// those of e4m3_rn_satfinite).
__device__ __forceinline__ uint32_t e4m3x4_rn(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// 16 values of pool row prow (pieces at ea and eb), in the pool's type.
// `split`: the pieces are halves of two E2M1 blocks whose other halves lie in
// the neighbouring lane.
template <typename T, int QUANT>
__device__ __forceinline__ void store_pool16(const WriteArgs& w, bool key, int64_t prow, int d, int ea, int eb,
                                             float (&x)[16], bool split, int u) {
  uint8_t* pool = static_cast<uint8_t*>(key ? w.pool_k : w.pool_v);
  if constexpr (QUANT == kQuantNone) {
    store_row_piece<T, 8>(reinterpret_cast<T*>(pool) + prow * d + ea, *reinterpret_cast<float(*)[8]>(x));
    store_row_piece<T, 8>(reinterpret_cast<T*>(pool) + prow * d + eb, *reinterpret_cast<float(*)[8]>(x + 8));
  } else {
    const float descale = key ? w.k_descale : w.v_descale;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], descale);
    if constexpr (QUANT == kQuantE4m3) {
      uint8_t* dst = pool + prow * d;
      *reinterpret_cast<uint2*>(dst + ea) =
          make_uint2(e4m3x4_rn(x[0], x[1], x[2], x[3]), e4m3x4_rn(x[4], x[5], x[6], x[7]));
      *reinterpret_cast<uint2*>(dst + eb) =
          make_uint2(e4m3x4_rn(x[8], x[9], x[10], x[11]), e4m3x4_rn(x[12], x[13], x[14], x[15]));
    } else {
      float va = 0.f, vb = 0.f;
      int na = 0, nb = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        va = fmaxf(va, fabsf(x[i]));
        vb = fmaxf(vb, fabsf(x[8 + i]));
        na |= x[i] != x[i];
        nb |= x[8 + i] != x[8 + i];
      }
      if (split) {
        const uint32_t mates = 3u << (threadIdx.x & 30);  // the two lanes of a block
        va = fmaxf(va, __shfl_xor_sync(mates, va, 1));
        vb = fmaxf(vb, __shfl_xor_sync(mates, vb, 1));
        na |= __shfl_xor_sync(mates, na, 1);
        nb |= __shfl_xor_sync(mates, nb, 1);
      } else {
        va = vb = fmaxf(va, vb);
        na = nb = na | nb;
      }
      const uint32_t sa = na ? 0x7Fu : e4m3_rn_satfinite(__fdiv_rn(va, 6.f));
      const uint32_t sb = nb ? 0x7Fu : e4m3_rn_satfinite(__fdiv_rn(vb, 6.f));
      uint32_t* dst = reinterpret_cast<uint32_t*>(pool + prow * (d / 2));
      dst[ea / 8] = fp4_codes8(x, sa);
      dst[eb / 8] = fp4_codes8(x + 8, sb);
      uint8_t* scales = pool + (key ? w.scale_off_k : w.scale_off_v) + prow * (d / 16);
      if (!split || (u & 1) == 0) {
        scales[ea / 16] = static_cast<uint8_t>(sa);
        if (split) scales[eb / 16] = static_cast<uint8_t>(sb);
      }
    }
  }
}

__device__ __forceinline__ void turn_pair(float& u, float& v, float c, float s) {
  const float f = u, g = v;
  u = __fadd_rn(__fmul_rn(f, c), -__fmul_rn(g, s));
  v = __fadd_rn(__fmul_rn(g, c), __fmul_rn(f, s));
}

struct RopeGeo {
  int units;             // pieces of 16 values a row
  int lanes;             // threads a unit of one token: they take rows lane, lane + lanes, ...
  int tokens_per_block;  // ... of that many tokens
};

template <typename T, int QUANT, int ROWS>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_pieces_kernel(const RopeArgs a, const RopeGeo geo) {
  pdl_trigger();
  pdl_wait();
  const WriteArgs& w = a.w;
  const int lane_row = threadIdx.x / geo.units;
  const int u = threadIdx.x - lane_row * geo.units;
  int t = blockIdx.x, lane = lane_row;
  if (geo.tokens_per_block > 1) {
    const int dt = lane_row / geo.lanes;
    t = t * geo.tokens_per_block + dt;
    lane -= dt * geo.lanes;
    if (dt >= geo.tokens_per_block) return;
  }
  if (lane >= geo.lanes || t >= w.num_tokens) return;
  const int nq = a.q != nullptr ? a.num_q_heads : 0;
  const int hkv = w.num_kv_heads;
  const int rows = nq + hkv * (w.pool_v != nullptr ? 2 : 1);
  const int r0 = blockIdx.y * geo.lanes * ROWS + lane;
  const int pos = __ldg(w.positions + t);
  if (pos < 0 || t >= __ldg(w.qo_indptr + w.num_rows)) return;  // padding token
  if (pos >= a.table_len) {
    if (r0 == 0 && u == 0) report(w.dev_status, CPATTN_DEV_POS_PAST_ROPE);
    return;
  }
  // pieces of a query or key row (a value row: u * 16, + 8)
  const int rot_units = a.rot_dim / 16;
  const bool turn = u < rot_units;
  int ea, eb;
  if (turn) {
    ea = a.rot_begin + (a.pairs ? u * 16 : u * 8);
    eb = a.pairs ? ea + 8 : ea + a.rot_dim / 2;
  } else {
    ea = (u - rot_units) * 16;
    if (ea >= a.rot_begin) ea += a.rot_dim;
    eb = ea + 8;
  }
  Piece16<T> raw[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int r = r0 + k * geo.lanes;
    if (r >= rows) continue;
    if (r < nq) {
      const T* src = static_cast<const T*>(a.q) + (static_cast<int64_t>(t) * nq + r) * a.head_dim;
      raw[k].load(src + ea, src + eb);
    } else if (r < nq + hkv) {
      const T* src = static_cast<const T*>(w.k_new) + (static_cast<int64_t>(t) * hkv + r - nq) * a.head_dim;
      raw[k].load(src + ea, src + eb);
    } else if (u * 16 < a.head_dim_v) {
      const T* src = static_cast<const T*>(w.v_new) + (static_cast<int64_t>(t) * hkv + r - nq - hkv) * a.head_dim_v;
      raw[k].load(src + u * 16, src + u * 16 + 8);
    }
  }
  float c[8], s[8];
  if (turn) {
    const float4* cs = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim + u * 8);
    const float4* sn = cs + a.rot_dim / 8;
    const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1), s0 = __ldg(sn), s1 = __ldg(sn + 1);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
  }
  // the token's slot, for threads with key or value rows
  int64_t row0 = -1;
  if (r0 + (ROWS - 1) * geo.lanes >= nq) {
    const int b = find_row(w.qo_indptr, w.num_rows, t);
    row0 = pool_row0(w, b, pos, u == 0);
  }
  const int ps_l = w.page_size / w.P;
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int r = r0 + k * geo.lanes;
    if (r >= rows) continue;
    const int kind = r < nq ? 0 : (r < nq + hkv ? 1 : 2);
    float x[16];
    raw[k].widen(x);
    if (kind == 2) {
      if (u * 16 < a.head_dim_v && row0 >= 0)
        store_pool16<T, QUANT>(w, false, row0 + static_cast<int64_t>(r - nq - hkv) * ps_l, a.head_dim_v, u * 16,
                               u * 16 + 8, x, false, u);
      continue;
    }
    if (turn) {
      // two loops, so that x stays in registers (a computed index would put it in local memory)
      if (a.pairs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(x[i], x[i + 8], c[i], s[i]);
      }
    }
    const int64_t row = static_cast<int64_t>(t) * (kind == 0 ? nq : hkv) + (kind == 0 ? r : r - nq);
    T* out = static_cast<T*>(kind == 0 ? a.q_out : a.k_out);
    if (out != nullptr) {
      store_row_piece<T, 8>(out + row * a.head_dim + ea, *reinterpret_cast<float(*)[8]>(x));
      store_row_piece<T, 8>(out + row * a.head_dim + eb, *reinterpret_cast<float(*)[8]>(x + 8));
    }
    if (kind == 1 && row0 >= 0)
      store_pool16<T, QUANT>(w, true, row0 + static_cast<int64_t>(r - nq) * ps_l, a.head_dim, ea, eb, x,
                             turn && !a.pairs, u);
  }
}

template <typename T, int QUANT, int ROWS>
static int launch_pieces(const RopeArgs& a, cudaStream_t s) {
  const int rows = (a.q != nullptr ? a.num_q_heads : 0) + a.w.num_kv_heads * (a.w.pool_v != nullptr ? 2 : 1);
  RopeGeo geo;
  geo.units = a.head_dim / 16;
  geo.lanes = kRopeThreads / geo.units;
  const int want = (rows + ROWS - 1) / ROWS;  // a thread takes up to ROWS rows
  if (geo.lanes > want) geo.lanes = want;
  geo.tokens_per_block = kRopeThreads / (geo.units * geo.lanes);
  const dim3 grid((a.w.num_tokens + geo.tokens_per_block - 1) / geo.tokens_per_block,
                  (rows + geo.lanes * ROWS - 1) / (geo.lanes * ROWS));
  if (grid.y > 65535) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  const int threads = (geo.tokens_per_block * geo.lanes * geo.units + 31) / 32 * 32;  // no idle warps
  return launch_pdl(rope_pieces_kernel<T, QUANT, ROWS>, grid, dim3(threads), 0, s, a, geo) == cudaSuccess
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}

template <typename T, int QUANT>
static int launch_rows(const RopeArgs& a, cudaStream_t s) {
  const int64_t per_token = (a.q != nullptr ? a.num_q_heads : 0) + a.w.num_kv_heads * (a.w.pool_v != nullptr ? 2 : 1);
  const int64_t blocks = (per_token * a.w.num_tokens + kRopeWarps - 1) / kRopeWarps;
  if (blocks > 0x7fffffff) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  const size_t smem = static_cast<size_t>(kRopeWarps) * a.head_dim * sizeof(float);
  auto kern = rope_rows_kernel<T, QUANT>;
  if (smem > 32 * 1024) {
    static std::atomic<int> smem_set[64];
    if (ensure_smem(kern, smem, smem_set) != cudaSuccess) return CPATTN_ERR_CUDA;
  }
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kRopeWarps * 32), smem, s, a) == cudaSuccess
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}

template <typename T, int QUANT>
static int launch_rope(const RopeArgs& a, cudaStream_t s) {
  // whole pieces for every row, and both lanes of a split E2M1 block in the same place of a warp
  const bool pieces = a.rot_dim % 16 == 0 && a.rot_begin % 16 == 0 && a.head_dim % 16 == 0 && a.head_dim_v % 16 == 0 &&
                      (QUANT != kQuantFp4 || a.pairs || a.rot_dim % 32 == 0);
  if (!pieces) return launch_rows<T, QUANT>(a, s);
  return a.w.num_tokens >= kRopeManyTokens ? launch_pieces<T, QUANT, sizeof(T) == 4 ? 2 : 4>(a, s)
                                           : launch_pieces<T, QUANT, 1>(a, s);
}

int launch_rope_kv_write(const RopeArgs& a, cudaStream_t s) {
  if (a.elem_bytes == 4) return launch_rope<float, kQuantNone>(a, s);
  switch (a.w.quant) {
    case kQuantNone: return launch_rope<__nv_bfloat16, kQuantNone>(a, s);
    case kQuantE4m3: return launch_rope<__nv_bfloat16, kQuantE4m3>(a, s);
    default: return launch_rope<__nv_bfloat16, kQuantFp4>(a, s);
  }
}

}  // namespace cpattn
