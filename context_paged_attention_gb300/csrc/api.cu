// C ABI of libcpattn (declared in include/cpattn.h): argument checks on the
// host, then the kernel launches.  Nothing here allocates, synchronises or
// keeps state between calls.
#include <algorithm>
#include <cstdint>

#include "cpattn.h"
#include "launch.h"

using namespace cpattn;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int dtype_bytes(int dtype) {
  if (dtype == CPATTN_DTYPE_BF16) return 2;
  if (dtype == CPATTN_DTYPE_FP32) return 4;
  return 0;
}

// Interleave size: 0 in the descriptor means 1 (plain striping).
int interleave_of(const cpattn_pool_desc* d) { return d->interleave > 1 ? d->interleave : 1; }

// Pool element type: kv_dtype 0 means the layer's dtype.
int kv_dtype_of(const cpattn_pool_desc* d) { return d->kv_dtype == 0 ? d->dtype : d->kv_dtype; }

bool is_fp8(const cpattn_pool_desc* d) { return kv_dtype_of(d) == CPATTN_DTYPE_FP8_E4M3; }
bool is_fp4(const cpattn_pool_desc* d) { return kv_dtype_of(d) == CPATTN_DTYPE_FP4_E2M1; }

// Bytes of a pool row of n values (E2M1: its codes, without the block scales).
int row_bytes(const cpattn_pool_desc* d, int n) {
  return is_fp4(d) ? n / 2 : (is_fp8(d) ? n : n * dtype_bytes(kv_dtype_of(d)));
}

// Rows of a pool tensor: [P][num_pages][num_kv_heads][page_size / P].
int64_t pool_rows(const cpattn_pool_desc* d) {
  return static_cast<int64_t>(d->num_pages) * d->num_kv_heads * d->page_size;
}

// Common descriptor checks.
int check_desc(const cpattn_pool_desc* d) {
  if (d == nullptr) return CPATTN_ERR_INVALID_ARG;
  if (d->P < 1 || d->page_size < 1 || d->interleave < 0 || d->page_size % (d->P * interleave_of(d)) != 0)
    return CPATTN_ERR_P_NOT_DIVIDING_PAGE_SIZE;
  if (d->num_pages < 1 || d->num_kv_heads < 1 || d->head_dim < 1 || d->head_dim_v < 1)
    return CPATTN_ERR_INVALID_ARG;
  const int eb = dtype_bytes(d->dtype);
  if (eb == 0) return CPATTN_ERR_INVALID_ARG;
  const int kt = kv_dtype_of(d);
  if (kt != d->dtype && kt != CPATTN_DTYPE_FP8_E4M3 && kt != CPATTN_DTYPE_FP4_E2M1) return CPATTN_ERR_INVALID_ARG;
  if (kt == CPATTN_DTYPE_FP8_E4M3 || kt == CPATTN_DTYPE_FP4_E2M1) {
    if (d->dtype != CPATTN_DTYPE_BF16) return CPATTN_ERR_UNSUPPORTED_SHAPE;
    const float ks = d->k_descale, vs = d->v_descale;
    if (!(ks > 0.f && ks <= 3.0e38f) || !(vs > 0.f && vs <= 3.0e38f)) return CPATTN_ERR_INVALID_ARG;
  }
  if ((d->head_dim * eb) % 16 != 0 || (d->head_dim_v * eb) % 16 != 0) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  if (kt == CPATTN_DTYPE_FP4_E2M1 && (d->head_dim % 32 != 0 || d->head_dim_v % 32 != 0))
    return CPATTN_ERR_UNSUPPORTED_SHAPE;
  if (row_bytes(d, d->head_dim) % 16 != 0 || row_bytes(d, d->head_dim_v) % 16 != 0)
    return CPATTN_ERR_UNSUPPORTED_SHAPE;
  if (d->head_dim_v > d->head_dim) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  return CPATTN_OK;
}

bool is_mla(const cpattn_pool_desc* d) { return d->head_dim_v != d->head_dim; }

}  // namespace

namespace {

// Output side of a partial launch: per-partner partials (o_part / lse_part)
// or, fused, the merged output.
struct FusedOut {
  int fused = 0;
  const float* extra_o = nullptr;
  const float* extra_lse = nullptr;
  void* out = nullptr;
  int out_bf16 = 0;
  float* lse_out = nullptr;
  const int32_t* row_order = nullptr;
};

// A score modification: null, or a cap that is 0 or within [1e-6, 1e30].
int check_mod(const cpattn_score_mod* m) {
  if (m == nullptr || m->softcap == 0.f) return CPATTN_OK;
  return m->softcap >= 1e-6f && m->softcap <= 1e30f ? CPATTN_OK : CPATTN_ERR_INVALID_ARG;
}

bool modifies(const cpattn_score_mod* m) { return m != nullptr && (m->softcap > 0.f || m->slopes != nullptr); }

WriteArgs write_args(const cpattn_pool_desc* desc, void* pool_k, void* pool_v, const void* k_new, const void* v_new,
                     const int32_t* positions, const int32_t* qo_indptr, int32_t num_rows, int32_t num_tokens,
                     const int32_t* kv_page_indptr, const int32_t* kv_page_indices, int32_t* dev_status) {
  const bool mla = is_mla(desc);
  const int eb = dtype_bytes(desc->dtype);
  WriteArgs a;
  a.pool_k = pool_k;
  a.pool_v = pool_v;
  a.k_new = k_new;
  a.v_new = v_new;
  a.positions = positions;
  a.qo_indptr = qo_indptr;
  a.page_indptr = kv_page_indptr;
  a.page_indices = kv_page_indices;
  a.dev_status = dev_status;
  a.P = desc->P;
  a.interleave = interleave_of(desc);
  a.page_size = desc->page_size;
  a.num_pages = desc->num_pages;
  a.num_kv_heads = desc->num_kv_heads;
  a.num_rows = num_rows;
  a.num_tokens = num_tokens;
  a.row_bytes_k = row_bytes(desc, desc->head_dim);
  a.row_bytes_v = mla ? 0 : row_bytes(desc, desc->head_dim_v);
  a.src_row_bytes_k = desc->head_dim * eb;
  a.src_row_bytes_v = mla ? 0 : desc->head_dim_v * eb;
  a.quant = is_fp4(desc) ? kQuantFp4 : (is_fp8(desc) ? kQuantE4m3 : kQuantNone);
  a.k_descale = desc->k_descale;
  a.v_descale = desc->v_descale;
  a.scale_off_k = pool_rows(desc) * a.row_bytes_k;
  a.scale_off_v = pool_rows(desc) * a.row_bytes_v;
  return a;
}

size_t partial_workspace(const cpattn_pool_desc* desc, int fused, int32_t num_q_heads, int32_t num_tokens,
                         int32_t max_kv_len) {
  if (check_desc(desc) != CPATTN_OK || num_q_heads < 1 || num_tokens < 0 || max_kv_len < 0) return 0;
  if (num_q_heads % desc->num_kv_heads != 0) return 0;
  if (is_fp4(desc) && max_kv_len > (1 << 30)) return 0;  // refused by the calls
  PartialPlan plan;
  if (!plan_partial(is_mla(desc), fused, is_fp4(desc), desc->P, interleave_of(desc), desc->page_size, desc->num_kv_heads,
                    num_q_heads, desc->head_dim, num_tokens, max_kv_len, dtype_bytes(desc->dtype), &plan))
    return 0;
  return plan.bytes();
}

int run_partial(const cpattn_pool_desc* desc, const void* pool_k, const void* pool_v, const void* q,
                int32_t num_q_heads, int32_t num_rows, int32_t num_tokens, const int32_t* qo_indptr,
                const int32_t* kv_len, int32_t max_kv_len, const int32_t* kv_page_indptr,
                const int32_t* kv_page_indices, float scale, float* o_part, float* lse_part, int lse_layout,
                const FusedOut& f, const cpattn_score_mod* mod, void* workspace, size_t workspace_bytes,
                int32_t* dev_status, cudaStream_t stream) {
  int st = check_desc(desc);
  if (st == CPATTN_OK) st = check_mod(mod);
  if (st != CPATTN_OK) return st;
  if (num_q_heads < 1 || num_rows < 0 || num_tokens < 0 || max_kv_len < 0) return CPATTN_ERR_INVALID_ARG;
  if (num_q_heads % desc->num_kv_heads != 0) return CPATTN_ERR_INVALID_ARG;
  if (qo_indptr == nullptr && num_tokens != num_rows) return CPATTN_ERR_INVALID_ARG;
  if (num_tokens == 0) return CPATTN_OK;
  const bool mla = is_mla(desc);
  if (pool_k == nullptr || q == nullptr || num_rows < 1 || kv_len == nullptr || kv_page_indptr == nullptr ||
      kv_page_indices == nullptr)
    return CPATTN_ERR_INVALID_ARG;
  if (!f.fused && (o_part == nullptr || lse_part == nullptr)) return CPATTN_ERR_INVALID_ARG;
  if (lse_layout != CPATTN_LSE_TOKEN_MAJOR && lse_layout != CPATTN_LSE_HEAD_MAJOR) return CPATTN_ERR_INVALID_ARG;
  if (!mla && pool_v == nullptr) return CPATTN_ERR_INVALID_ARG;
  if (mla && pool_v != nullptr && pool_v != pool_k) return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(pool_k) || !aligned16(pool_v) || !aligned16(q) || !aligned16(o_part) || !aligned16(workspace))
    return CPATTN_ERR_MISALIGNED;
  if (mla && desc->dtype != CPATTN_DTYPE_BF16) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  // E4M3 and E2M1 pools: GQA (the MLA kernel reads bf16 latent rows only)
  if ((is_fp8(desc) || is_fp4(desc) || modifies(mod)) && mla) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  // the decode kernel over codes keeps pool rows as 32-bit values (2^32 - 1 rows are 137 GB of E2M1 codes at D 64)
  if ((is_fp4(desc) || (is_fp8(desc) && modifies(mod))) && pool_rows(desc) >= 0xffffffffLL)
    return CPATTN_ERR_UNSUPPORTED_SHAPE;
  // multi-token rows over a pool of 16-bit or narrower rows: the kernel's copy warps pass pool row
  // indices as 32-bit values (checked here, before the one-token rows' launch)
  if (!mla && qo_indptr != nullptr && (!is_fp8(desc) || modifies(mod)) && pool_rows(desc) >= (int64_t{1} << 31))
    return CPATTN_ERR_UNSUPPORTED_SHAPE;
  // run and stripe lengths are rounded up in 32 bits
  if ((is_fp4(desc) || modifies(mod)) && max_kv_len > (1 << 30)) return CPATTN_ERR_UNSUPPORTED_SHAPE;

  PartialPlan plan;
  if (!plan_partial(mla, f.fused, is_fp4(desc), desc->P, interleave_of(desc), desc->page_size, desc->num_kv_heads, num_q_heads,
                    desc->head_dim, num_tokens, max_kv_len, dtype_bytes(desc->dtype), &plan))
    return CPATTN_ERR_UNSUPPORTED_SHAPE;
  const size_t need = plan.bytes();
  if (workspace == nullptr || workspace_bytes < need) return CPATTN_ERR_WORKSPACE_TOO_SMALL;

  // workspace: chunk partials, chunk LSEs, partner partials, partner LSEs
  // (fused), then the two ticket arrays side by side (one memset)
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PartialArgs a;
  size_t off = 0;
  a.ws_o = reinterpret_cast<float*>(ws + off);
  off += al(plan.ws_o_floats * 4);
  a.ws_lse = reinterpret_cast<float*>(ws + off);
  off += al(plan.ws_lse_floats * 4);
  float* ws_part = reinterpret_cast<float*>(ws + off);
  off += al(plan.ws_part_floats * 4);
  float* ws_part_lse = reinterpret_cast<float*>(ws + off);
  off += al(plan.ws_part_lse_floats * 4);
  a.ws_cnt = reinterpret_cast<int32_t*>(ws + off);
  const size_t cnt_bytes = al(plan.ws_cnt_ints * 4);
  a.ws_pair = reinterpret_cast<int32_t*>(ws + off + cnt_bytes);
  const size_t ticket_bytes = cnt_bytes + plan.ws_pair_ints * 4;
  if (f.fused) {
    o_part = ws_part;
    lse_part = ws_part_lse;
  }
  a.pool_k = pool_k;
  a.pool_v = mla ? pool_k : pool_v;
  a.q = q;
  a.o_part = o_part;
  a.lse_part = lse_part;
  // LSE of (partner, token, head): [P][T][Hq], or [P][Hq][T] (FlashAttention's [H, B] per partner);
  // the partner partials of fused calls are internal and token-major
  const int64_t TH = static_cast<int64_t>(num_tokens) * num_q_heads;
  const bool head_major = !f.fused && lse_layout == CPATTN_LSE_HEAD_MAJOR;
  a.lse_sp = TH;
  a.lse_st = head_major ? 1 : num_q_heads;
  a.lse_sh = head_major ? num_tokens : 1;
  a.qo_indptr = qo_indptr;
  a.kv_len = kv_len;
  a.page_indptr = kv_page_indptr;
  a.page_indices = kv_page_indices;
  a.dev_status = dev_status;
  a.P = desc->P;
  a.interleave = interleave_of(desc);
  a.page_size = desc->page_size;
  a.ps_l = desc->page_size / desc->P;
  a.ps_shift = -1;
  for (int sh = 0; sh < 31; ++sh)
    if ((1 << sh) == a.ps_l) a.ps_shift = sh;
  a.num_pages = desc->num_pages;
  a.num_kv_heads = desc->num_kv_heads;
  a.num_q_heads = num_q_heads;
  a.head_dim = desc->head_dim;
  a.head_dim_v = desc->head_dim_v;
  a.num_rows = num_rows;
  a.num_tokens = num_tokens;
  a.max_kv_len = max_kv_len;
  a.seg = plan.seg;
  a.chunk = plan.chunk;
  a.max_chunks = plan.max_chunks;
  a.run = plan.run;
  a.max_runs = plan.max_runs;
  a.ws_run_o = ws_part;
  a.ws_run_lse = ws_part_lse;
  if (f.fused && is_fp8(desc) && modifies(mod)) {
    // their pieces lie where the chunks' (or the partners') partials would: a
    // row of L keys has ceil(L / run) of them, and there is room for P * max_chunks
    const int room = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(desc->P) * plan.max_chunks, 1 << 20));
    const int run = std::max(codes_run(desc->page_size, desc->num_kv_heads, num_tokens, max_kv_len), (max_kv_len + room - 1) / room);
    a.run = (run + desc->page_size - 1) / desc->page_size * desc->page_size;
    a.max_runs = max_kv_len > 0 ? (max_kv_len + a.run - 1) / a.run : 1;
    a.ws_run_o = plan.max_chunks > 1 ? a.ws_o : ws_part;
    a.ws_run_lse = plan.max_chunks > 1 ? a.ws_lse : ws_part_lse;
  }
  a.scale = scale;
  a.kv_fp8 = is_fp8(desc);
  a.kv_fp4 = is_fp4(desc);
  a.scale_off = pool_rows(desc) * row_bytes(desc, desc->head_dim);
  a.k_descale = desc->k_descale;
  a.v_descale = desc->v_descale;
  a.has_mod = modifies(mod);
  a.softcap = a.has_mod ? mod->softcap : 0.f;
  a.slopes = a.has_mod ? mod->slopes : nullptr;
  a.q_pos = a.has_mod ? mod->positions : nullptr;
  a.q_pos_own = qo_indptr == nullptr;
  a.fused = f.fused;
  a.extra_o = f.extra_o;
  a.extra_lse = f.extra_lse;
  a.out = f.out;
  a.out_bf16 = f.out_bf16;
  a.lse_out = f.lse_out;
  a.row_order = f.row_order;

  // tickets start from zero (each call's last arrivals also reset them); fused decode calls that take whole page runs
  // use them only for rows of several runs
  const bool by_runs = f.fused && qo_indptr == nullptr && a.max_runs > 0 && (a.kv_fp4 || a.has_mod);
  if (by_runs ? a.max_runs > 1 : (plan.max_chunks > 1 || f.fused)) {
    if (cudaMemsetAsync(a.ws_cnt, 0, ticket_bytes, stream) != cudaSuccess) return CPATTN_ERR_CUDA;
  }
  cudaError_t err = cudaSuccess;
  if (mla) return launch_mla_partial(a, stream, &err);
  return launch_gqa_partial(a, desc->dtype == CPATTN_DTYPE_BF16, stream, &err);
}

}  // namespace

extern "C" {

int cpattn_version(void) { return CPATTN_VERSION; }

const char* cpattn_status_string(int status) {
  switch (status) {
    case CPATTN_OK: return "ok";
    case CPATTN_ERR_INVALID_ARG: return "invalid argument";
    case CPATTN_ERR_P_NOT_DIVIDING_PAGE_SIZE: return "P and interleave must be >= 1 and P * interleave divide page_size";
    case CPATTN_ERR_UNSUPPORTED_SHAPE: return "unsupported shape (head dims / group size)";
    case CPATTN_ERR_MISALIGNED: return "device pointer not 16-byte aligned";
    case CPATTN_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case CPATTN_ERR_CUDA: return "CUDA launch failed";
    default: return "unknown status";
  }
}

size_t cpattn_pool_bytes(const cpattn_pool_desc* d, int which_v) {
  if (check_desc(d) != CPATTN_OK) return 0;
  const int n = which_v ? d->head_dim_v : d->head_dim;
  return static_cast<size_t>(pool_rows(d)) * (row_bytes(d, n) + (is_fp4(d) ? n / 16 : 0));
}

int cp_kv_write(const cpattn_pool_desc* desc, void* pool_k, void* pool_v, const void* k_new, const void* v_new,
                const int32_t* positions, const int32_t* qo_indptr, int32_t num_rows, int32_t num_tokens,
                const int32_t* kv_page_indptr, const int32_t* kv_page_indices, int32_t* dev_status,
                cudaStream_t stream) {
  int st = check_desc(desc);
  if (st != CPATTN_OK) return st;
  if (num_rows < 0 || num_tokens < 0) return CPATTN_ERR_INVALID_ARG;
  if (num_tokens == 0) return CPATTN_OK;
  const bool mla = is_mla(desc);
  if (pool_k == nullptr || k_new == nullptr || positions == nullptr || qo_indptr == nullptr ||
      kv_page_indptr == nullptr || kv_page_indices == nullptr || num_rows < 1)
    return CPATTN_ERR_INVALID_ARG;
  if (!mla && (pool_v == nullptr || v_new == nullptr)) return CPATTN_ERR_INVALID_ARG;
  if (mla && (pool_v != nullptr || v_new != nullptr)) return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(pool_k) || !aligned16(pool_v) || !aligned16(k_new) || !aligned16(v_new))
    return CPATTN_ERR_MISALIGNED;
  const WriteArgs a = write_args(desc, pool_k, pool_v, k_new, v_new, positions, qo_indptr, num_rows, num_tokens,
                                 kv_page_indptr, kv_page_indices, dev_status);
  return launch_kv_write(a, stream) == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

int cp_rope_kv_write(const cpattn_pool_desc* desc, void* pool_k, void* pool_v, const void* q, const void* k_new,
                     const void* v_new, int32_t num_q_heads, const int32_t* positions, const int32_t* qo_indptr,
                     int32_t num_rows, int32_t num_tokens, const int32_t* kv_page_indptr,
                     const int32_t* kv_page_indices, const float* cos_sin, int32_t table_len, int32_t rot_begin,
                     int32_t rot_dim, int32_t style, void* q_out, void* k_out, int32_t* dev_status,
                     cudaStream_t stream) {
  const int st = check_desc(desc);
  if (st != CPATTN_OK) return st;
  if (num_rows < 0 || num_tokens < 0 || table_len < 1) return CPATTN_ERR_INVALID_ARG;
  if (style != CPATTN_ROPE_HALVES && style != CPATTN_ROPE_PAIRS) return CPATTN_ERR_INVALID_ARG;
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_begin < 0 || rot_begin > desc->head_dim - rot_dim)
    return CPATTN_ERR_INVALID_ARG;
  // rows pass through shared memory as float32, 64 KB a CTA at most
  if (desc->head_dim > 2048) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  if ((q == nullptr) != (q_out == nullptr) || (q != nullptr && num_q_heads < 1)) return CPATTN_ERR_INVALID_ARG;
  if (num_tokens == 0) return CPATTN_OK;
  const bool mla = is_mla(desc);
  if (pool_k == nullptr || k_new == nullptr || positions == nullptr || qo_indptr == nullptr ||
      kv_page_indptr == nullptr || kv_page_indices == nullptr || cos_sin == nullptr || num_rows < 1)
    return CPATTN_ERR_INVALID_ARG;
  if (!mla && (pool_v == nullptr || v_new == nullptr)) return CPATTN_ERR_INVALID_ARG;
  if (mla && (pool_v != nullptr || v_new != nullptr)) return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(pool_k) || !aligned16(pool_v) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q) ||
      !aligned16(q_out) || !aligned16(k_out) || !aligned16(cos_sin))
    return CPATTN_ERR_MISALIGNED;
  RopeArgs a;
  a.w = write_args(desc, pool_k, pool_v, k_new, v_new, positions, qo_indptr, num_rows, num_tokens, kv_page_indptr,
                   kv_page_indices, dev_status);
  a.q = q;
  a.q_out = q_out;
  a.k_out = k_out;
  a.cos_sin = cos_sin;
  a.num_q_heads = num_q_heads;
  a.head_dim = desc->head_dim;
  a.head_dim_v = mla ? 0 : desc->head_dim_v;
  a.elem_bytes = dtype_bytes(desc->dtype);
  a.rot_begin = rot_begin;
  a.rot_dim = rot_dim;
  a.pairs = style == CPATTN_ROPE_PAIRS;
  a.table_len = table_len;
  return launch_rope_kv_write(a, stream);
}

size_t cp_paged_attn_workspace_bytes(const cpattn_pool_desc* desc, int32_t num_q_heads, int32_t num_tokens,
                                     int32_t max_kv_len) {
  return partial_workspace(desc, 0, num_q_heads, num_tokens, max_kv_len);
}

size_t cp_paged_attn_fused_workspace_bytes(const cpattn_pool_desc* desc, int32_t num_q_heads, int32_t num_tokens,
                                           int32_t max_kv_len) {
  return partial_workspace(desc, 1, num_q_heads, num_tokens, max_kv_len);
}

int cp_paged_attn_partial(const cpattn_pool_desc* desc, const void* pool_k, const void* pool_v, const void* q,
                          int32_t num_q_heads, int32_t num_rows, int32_t num_tokens, const int32_t* qo_indptr,
                          const int32_t* kv_len, int32_t max_kv_len, const int32_t* kv_page_indptr,
                          const int32_t* kv_page_indices, float scale, float* o_part, float* lse_part,
                          void* workspace, size_t workspace_bytes, int32_t* dev_status, cudaStream_t stream) {
  FusedOut none;
  return run_partial(desc, pool_k, pool_v, q, num_q_heads, num_rows, num_tokens, qo_indptr, kv_len, max_kv_len,
                     kv_page_indptr, kv_page_indices, scale, o_part, lse_part, CPATTN_LSE_TOKEN_MAJOR, none,
                     nullptr, workspace, workspace_bytes, dev_status, stream);
}

int cp_paged_attn_partial_ex(const cpattn_pool_desc* desc, const void* pool_k, const void* pool_v, const void* q,
                             int32_t num_q_heads, int32_t num_rows, int32_t num_tokens, const int32_t* qo_indptr,
                             const int32_t* kv_len, int32_t max_kv_len, const int32_t* kv_page_indptr,
                             const int32_t* kv_page_indices, float scale, float* o_part, float* lse_part,
                             int32_t lse_layout, const int32_t* row_order, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, cudaStream_t stream) {
  return cp_paged_attn_partial_mod(desc, pool_k, pool_v, q, num_q_heads, num_rows, num_tokens, qo_indptr, kv_len,
                                   max_kv_len, kv_page_indptr, kv_page_indices, scale, o_part, lse_part, lse_layout,
                                   row_order, nullptr, workspace, workspace_bytes, dev_status, stream);
}

int cp_paged_attn_partial_mod(const cpattn_pool_desc* desc, const void* pool_k, const void* pool_v, const void* q,
                              int32_t num_q_heads, int32_t num_rows, int32_t num_tokens, const int32_t* qo_indptr,
                              const int32_t* kv_len, int32_t max_kv_len, const int32_t* kv_page_indptr,
                              const int32_t* kv_page_indices, float scale, float* o_part, float* lse_part,
                              int32_t lse_layout, const int32_t* row_order, const cpattn_score_mod* mod,
                              void* workspace, size_t workspace_bytes, int32_t* dev_status, cudaStream_t stream) {
  FusedOut none;
  none.row_order = qo_indptr == nullptr ? row_order : nullptr;
  return run_partial(desc, pool_k, pool_v, q, num_q_heads, num_rows, num_tokens, qo_indptr, kv_len, max_kv_len,
                     kv_page_indptr, kv_page_indices, scale, o_part, lse_part, lse_layout, none, mod, workspace,
                     workspace_bytes, dev_status, stream);
}

int cp_paged_attn_fused(const cpattn_pool_desc* desc, const void* pool_k, const void* pool_v, const void* q,
                        int32_t num_q_heads, int32_t num_rows, int32_t num_tokens, const int32_t* qo_indptr,
                        const int32_t* kv_len, int32_t max_kv_len, const int32_t* kv_page_indptr,
                        const int32_t* kv_page_indices, const int32_t* row_order, float scale,
                        const float* extra_o, const float* extra_lse,
                        int32_t out_dtype, void* out, float* lse_out, void* workspace, size_t workspace_bytes,
                        int32_t* dev_status, cudaStream_t stream) {
  return cp_paged_attn_fused_mod(desc, pool_k, pool_v, q, num_q_heads, num_rows, num_tokens, qo_indptr, kv_len,
                                 max_kv_len, kv_page_indptr, kv_page_indices, row_order, scale, extra_o, extra_lse,
                                 out_dtype, out, lse_out, nullptr, workspace, workspace_bytes, dev_status, stream);
}

int cp_paged_attn_fused_mod(const cpattn_pool_desc* desc, const void* pool_k, const void* pool_v, const void* q,
                            int32_t num_q_heads, int32_t num_rows, int32_t num_tokens, const int32_t* qo_indptr,
                            const int32_t* kv_len, int32_t max_kv_len, const int32_t* kv_page_indptr,
                            const int32_t* kv_page_indices, const int32_t* row_order, float scale,
                            const float* extra_o, const float* extra_lse, int32_t out_dtype, void* out, float* lse_out,
                            const cpattn_score_mod* mod, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                            cudaStream_t stream) {
  const int st = check_desc(desc);
  if (st != CPATTN_OK) return st;
  if (out_dtype != CPATTN_DTYPE_BF16 && out_dtype != CPATTN_DTYPE_FP32) return CPATTN_ERR_INVALID_ARG;
  if ((extra_o == nullptr) != (extra_lse == nullptr)) return CPATTN_ERR_INVALID_ARG;
  if (num_tokens > 0 && out == nullptr) return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(extra_o)) return CPATTN_ERR_MISALIGNED;
  if (out_dtype == CPATTN_DTYPE_BF16 && (desc->head_dim_v % 8) != 0) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  FusedOut f;
  f.fused = 1;
  f.extra_o = extra_o;
  f.extra_lse = extra_lse;
  f.out = out;
  f.out_bf16 = out_dtype == CPATTN_DTYPE_BF16;
  f.lse_out = lse_out;
  f.row_order = qo_indptr == nullptr ? row_order : nullptr;
  return run_partial(desc, pool_k, pool_v, q, num_q_heads, num_rows, num_tokens, qo_indptr, kv_len, max_kv_len,
                     kv_page_indptr, kv_page_indices, scale, nullptr, nullptr, CPATTN_LSE_TOKEN_MAJOR, f, mod, workspace,
                     workspace_bytes, dev_status, stream);
}

int own_token_attn(const void* q, const void* k_new, const void* v_new, int32_t num_q_heads, int32_t num_kv_heads,
                   int32_t head_dim, int32_t head_dim_v, int32_t dtype, const int32_t* qo_indptr,
                   int32_t num_rows_bucket, int32_t num_real_rows, int32_t num_tokens, int32_t max_q_len,
                   float scale, float* o_own, float* lse_own, cudaStream_t stream) {
  return own_token_attn_mod(q, k_new, v_new, num_q_heads, num_kv_heads, head_dim, head_dim_v, dtype, qo_indptr,
                            num_rows_bucket, num_real_rows, num_tokens, max_q_len, scale, nullptr, o_own, lse_own,
                            stream);
}

int own_token_attn_mod(const void* q, const void* k_new, const void* v_new, int32_t num_q_heads, int32_t num_kv_heads,
                       int32_t head_dim, int32_t head_dim_v, int32_t dtype, const int32_t* qo_indptr,
                       int32_t num_rows_bucket, int32_t num_real_rows, int32_t num_tokens, int32_t max_q_len,
                       float scale, const cpattn_score_mod* mod, float* o_own, float* lse_own, cudaStream_t stream) {
  const int eb = dtype_bytes(dtype);
  if (eb == 0 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0 || num_tokens < 0 ||
      num_rows_bucket < 1 || num_real_rows < 0 || num_real_rows > num_rows_bucket || max_q_len < 0)
    return CPATTN_ERR_INVALID_ARG;
  // MLA: one latent head, keys of 576 values whose first 512 are the value (v_new NULL)
  const bool mla = num_kv_heads == 1 && head_dim == 576 && head_dim_v == 512;
  if (check_mod(mod) != CPATTN_OK) return CPATTN_ERR_INVALID_ARG;
  if (mla ? (dtype != CPATTN_DTYPE_BF16 || v_new != nullptr || modifies(mod)) : head_dim != head_dim_v)
    return CPATTN_ERR_UNSUPPORTED_SHAPE;
  if (num_tokens == 0) return CPATTN_OK;
  if (q == nullptr || k_new == nullptr || qo_indptr == nullptr || o_own == nullptr || lse_own == nullptr)
    return CPATTN_ERR_INVALID_ARG;
  if (v_new == nullptr) v_new = k_new;  // value = prefix of the key row
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(o_own)) return CPATTN_ERR_MISALIGNED;
  OwnArgs a;
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.o_own = o_own;
  a.lse_own = lse_own;
  a.qo_indptr = qo_indptr;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.num_rows_bucket = num_rows_bucket;
  a.num_real_rows = num_real_rows;
  a.num_tokens = num_tokens;
  a.max_q_len = max_q_len;
  a.scale = scale;
  a.has_mod = modifies(mod);
  a.softcap = a.has_mod ? mod->softcap : 0.f;
  a.slopes = a.has_mod ? mod->slopes : nullptr;
  cudaError_t err = cudaSuccess;
  return launch_own_token(a, dtype == CPATTN_DTYPE_BF16, stream, &err);
}

int lse_merge(int32_t num_partials, const float* o_parts, const float* lse_parts, int64_t stride_o,
              int64_t stride_lse, int32_t num_tokens, int32_t num_heads, int32_t head_dim_v, int32_t out_dtype,
              void* out, float* lse_out, cudaStream_t stream) {
  if (num_partials < 1 || num_tokens < 0 || num_heads < 1 || head_dim_v < 4 || head_dim_v % 4 != 0)
    return CPATTN_ERR_INVALID_ARG;
  if (out_dtype != CPATTN_DTYPE_BF16 && out_dtype != CPATTN_DTYPE_FP32) return CPATTN_ERR_INVALID_ARG;
  if (num_tokens == 0) return CPATTN_OK;
  if (o_parts == nullptr || lse_parts == nullptr || out == nullptr) return CPATTN_ERR_INVALID_ARG;
  const int64_t per_o = static_cast<int64_t>(num_tokens) * num_heads * head_dim_v;
  const int64_t per_l = static_cast<int64_t>(num_tokens) * num_heads;
  if (num_partials > 1 && (stride_o < per_o || stride_lse < per_l)) return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(o_parts) || !aligned16(out) || (stride_o % 4) != 0) return CPATTN_ERR_MISALIGNED;
  if (out_dtype == CPATTN_DTYPE_BF16 && (head_dim_v % 8) != 0) return CPATTN_ERR_UNSUPPORTED_SHAPE;
  MergeArgs a;
  a.num_partials = num_partials;
  a.o_parts = o_parts;
  a.lse_parts = lse_parts;
  a.stride_o = stride_o;
  a.stride_lse = stride_lse;
  a.num_tokens = num_tokens;
  a.num_heads = num_heads;
  a.head_dim_v = head_dim_v;
  a.out_bf16 = out_dtype == CPATTN_DTYPE_BF16;
  a.out = out;
  a.lse_out = lse_out;
  return launch_lse_merge(a, stream) == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

int lse_merge_views(int32_t num_views, const cpattn_partial_view* views, int32_t num_tokens, int32_t num_heads,
                    int32_t head_dim_v, int32_t out_dtype, void* out, int64_t out_stride_token,
                    int64_t out_stride_head, float* lse_out, int64_t lse_out_stride_token,
                    int64_t lse_out_stride_head, cudaStream_t stream) {
  if (num_views < 1 || num_views > CPATTN_MAX_MERGE_VIEWS || views == nullptr || num_tokens < 0 || num_heads < 1 ||
      head_dim_v < 4 || head_dim_v % 4 != 0)
    return CPATTN_ERR_INVALID_ARG;
  if (out_dtype != CPATTN_DTYPE_BF16 && out_dtype != CPATTN_DTYPE_FP32) return CPATTN_ERR_INVALID_ARG;
  if (num_tokens == 0) return CPATTN_OK;
  if (out == nullptr) return CPATTN_ERR_INVALID_ARG;
  // 16-byte row starts: every row pointer and row stride a multiple of 4 elements
  if (!aligned16(out) || out_stride_token % 4 != 0 || out_stride_head % 4 != 0) return CPATTN_ERR_MISALIGNED;
  MergeViewArgs a;
  a.n = num_views;
  for (int i = 0; i < num_views; ++i) {
    const cpattn_partial_view& v = views[i];
    if (v.o == nullptr || v.lse == nullptr) return CPATTN_ERR_INVALID_ARG;
    if (!aligned16(v.o) || v.o_stride_token % 4 != 0 || v.o_stride_head % 4 != 0) return CPATTN_ERR_MISALIGNED;
    a.v[i].o = v.o;
    a.v[i].lse = v.lse;
    a.v[i].o_st = v.o_stride_token;
    a.v[i].o_sh = v.o_stride_head;
    a.v[i].lse_st = v.lse_stride_token;
    a.v[i].lse_sh = v.lse_stride_head;
  }
  a.num_tokens = num_tokens;
  a.num_heads = num_heads;
  a.head_dim_v = head_dim_v;
  a.out_bf16 = out_dtype == CPATTN_DTYPE_BF16;
  a.out = out;
  a.out_st = out_stride_token;
  a.out_sh = out_stride_head;
  a.lse_out = lse_out;
  a.lse_out_st = lse_out_stride_token;
  a.lse_out_sh = lse_out_stride_head;
  return launch_lse_merge_views(a, stream) == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

}  // extern "C"
