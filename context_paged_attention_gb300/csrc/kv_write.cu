// cp_kv_write: copy a step's new K/V rows into the P-way striped paged pool.
//
// Placement (mstar PR #1124 "Context / Sequence Parallel 1/5", description):
// offset off of a logical page belongs to partner off % P at physical slot
// off / P of the same page id.  With an interleave size I (vLLM's
// cp_kv_cache_interleave_size), runs of I offsets go together: partner
// (off / I) % P, physical slot (off / (I * P)) * I + off % I.  The review thread of that PR shows the failure
// this kernel must avoid: taking the slot at the logical page size, which makes
// every partner write every token at offsets up to page_size - 1.
//
// One thread moves one 16-byte chunk of one (token, KV head) row; the chunks of
// a row are adjacent threads, so both the read of k_new and the write into the
// pool are coalesced 16-byte accesses.
#include "kv_quant.cuh"

namespace cpattn {

// E4M3 codes of 16 bf16 values (byte offset src_off of src, chunk c) divided
// by the descale: IEEE float32 quotient, then e4m3_rn_satfinite.
__device__ __forceinline__ void store_fp8_chunk(const void* src, int64_t src_off, void* dst, int64_t dst_off, int c,
                                                float descale) {
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(src) + src_off) + 2 * c;
  const uint4 w0 = __ldg(s), w1 = __ldg(s + 1);
  const uint32_t in[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t pair = in[2 * i + j];
      const float lo = __fdiv_rn(bf16_lo(pair), descale);
      const float hi = __fdiv_rn(bf16_hi(pair), descale);
      const uint32_t b0 = e4m3_rn_satfinite(lo);
      const uint32_t b1 = e4m3_rn_satfinite(hi);
      word |= (b0 | (b1 << 8)) << (16 * j);
    }
    out[i] = word;
  }
  *(reinterpret_cast<uint4*>(static_cast<uint8_t*>(dst) + dst_off) + c) = make_uint4(out[0], out[1], out[2], out[3]);
}

// Block c (16 values) of one E2M1 row of nblk blocks from 16 bf16 values.
__device__ __forceinline__ void store_fp4_block(const void* src, int64_t src_off, void* pool, int64_t scale_off,
                                                int64_t prow, int nblk, int c, float descale) {
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(src) + src_off) + 2 * c;
  float x[16];
  Chunk16<__nv_bfloat16>::widen(__ldg(s), x);
  Chunk16<__nv_bfloat16>::widen(__ldg(s + 1), x + 8);
  uint2 codes;
  uint32_t scale;
  fp4_encode_block(x, descale, codes, scale);
  uint8_t* p = static_cast<uint8_t*>(pool);
  *reinterpret_cast<uint2*>(p + (prow * nblk + c) * 8) = codes;
  p[scale_off + prow * nblk + c] = static_cast<uint8_t>(scale);
}

__global__ void __launch_bounds__(256) kv_write_kernel(const WriteArgs a, int chunks_per_row) {
  pdl_trigger();
  pdl_wait();
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t per_token = static_cast<int64_t>(a.num_kv_heads) * chunks_per_row;
  const int64_t total = per_token * a.num_tokens;
  if (gid >= total) return;
  const int t = static_cast<int>(gid / per_token);
  const int rem = static_cast<int>(gid - static_cast<int64_t>(t) * per_token);
  const int h = rem / chunks_per_row;
  const int c = rem - h * chunks_per_row;

  const int b = row_of_token(a.qo_indptr, a.num_rows, t);
  if (b < 0) return;  // padding token past the last row
  const int pos = __ldg(a.positions + t);
  if (pos < 0) return;  // padding token
  const int64_t row0 = pool_row0(a, b, pos, c == 0 && h == 0);
  if (row0 < 0) return;
  const int64_t prow = row0 + static_cast<int64_t>(h) * (a.page_size / a.P);
  const int64_t srow = static_cast<int64_t>(t) * a.num_kv_heads + h;

  if (a.quant == kQuantFp4) {
    // a block of 16 values: 8 bytes of codes, one scale behind the pool's codes
    const int nblk_k = a.row_bytes_k / 8, nblk_v = a.row_bytes_v / 8;
    if (c < nblk_k) store_fp4_block(a.k_new, srow * a.src_row_bytes_k, a.pool_k, a.scale_off_k, prow, nblk_k, c, a.k_descale);
    if (a.pool_v != nullptr && c < nblk_v)
      store_fp4_block(a.v_new, srow * a.src_row_bytes_v, a.pool_v, a.scale_off_v, prow, nblk_v, c, a.v_descale);
    return;
  }
  if (a.quant == kQuantE4m3) {
    // 16 codes of the pool row from 16 bf16 values of the new row
    if (c * 16 < a.row_bytes_k) store_fp8_chunk(a.k_new, srow * a.src_row_bytes_k, a.pool_k, prow * a.row_bytes_k, c,
                                               a.k_descale);
    if (a.pool_v != nullptr && c * 16 < a.row_bytes_v)
      store_fp8_chunk(a.v_new, srow * a.src_row_bytes_v, a.pool_v, prow * a.row_bytes_v, c, a.v_descale);
    return;
  }
  if (c * 16 < a.row_bytes_k) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.k_new) +
                                                      srow * a.row_bytes_k) + c;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.pool_k) + prow * a.row_bytes_k) + c;
    *dst = __ldg(src);
  }
  if (a.pool_v != nullptr && c * 16 < a.row_bytes_v) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.v_new) +
                                                      srow * a.row_bytes_v) + c;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.pool_v) + prow * a.row_bytes_v) + c;
    *dst = __ldg(src);
  }
}

cudaError_t launch_kv_write(const WriteArgs& a, cudaStream_t s) {
  const int rb = a.row_bytes_k > a.row_bytes_v ? a.row_bytes_k : a.row_bytes_v;
  const int chunks = a.quant == kQuantFp4 ? rb / 8 : rb / 16;  // E2M1: one thread a block of 16 values
  const int64_t total = static_cast<int64_t>(a.num_tokens) * a.num_kv_heads * chunks;
  if (total == 0) return cudaSuccess;
  const int threads = 256;
  const int64_t blocks = (total + threads - 1) / threads;
  return launch_pdl(kv_write_kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, s, a, chunks);
}

}  // namespace cpattn
