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
constexpr int kRopeMaxDim = 2048;  // head_dim staged in shared memory (64 KB a CTA)

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

template <typename T, int QUANT>
static int launch_rows(const RopeArgs& a, cudaStream_t s) {
  const int64_t per_token = (a.q != nullptr ? a.num_q_heads : 0) + a.w.num_kv_heads * (a.w.pool_v != nullptr ? 2 : 1);
  const int64_t blocks = (per_token * a.w.num_tokens + kRopeWarps - 1) / kRopeWarps;
  if (a.head_dim > kRopeMaxDim || blocks > 0x7fffffff) return CPATTN_ERR_UNSUPPORTED_SHAPE;
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

int launch_rope_kv_write(const RopeArgs& a, cudaStream_t s) {
  if (a.elem_bytes == 4) return launch_rows<float, kQuantNone>(a, s);
  switch (a.w.quant) {
    case kQuantNone: return launch_rows<__nv_bfloat16, kQuantNone>(a, s);
    case kQuantE4m3: return launch_rows<__nv_bfloat16, kQuantE4m3>(a, s);
    default: return launch_rows<__nv_bfloat16, kQuantFp4>(a, s);
  }
}

}  // namespace cpattn
