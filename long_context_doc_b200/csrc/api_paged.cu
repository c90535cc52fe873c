// api_paged.cu - the extern "C" boundary of the paged local context (declared in
// include/msa.h): argument validation, workspace sizing and launches, as api.cu.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/msa.h"
#include "common.cuh"
#include "kernels.cuh"

namespace {

msa_status fail(msa_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
msa_status fail(msa_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  msa::set_last_error(buf);
  return s;
}

msa_status done(cudaError_t e, const char* what) {
  if (e != cudaSuccess)
    return fail(MSA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  msa::set_last_error("");
  return MSA_OK;
}

#define REQUIRE(cond, status, ...) \
  do {                             \
    if (!(cond)) return fail(status, __VA_ARGS__); \
  } while (0)

constexpr size_t kHeader = 256;
constexpr int32_t kMinPage = 16, kMaxHeads = 1024;
constexpr int32_t kMaxQueryHeads = 1 << 20;  // offsets within a row of Q are 32-bit

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t esize(int dtype) { return dtype == MSA_BF16 ? 2 : 4; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    return 148;
  return n;
}

int log2i(int32_t x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

msa_status check_pool(int32_t page_size, int32_t n_pages, int32_t max_pages, int32_t n_req) {
  REQUIRE(page_size >= kMinPage && page_size <= (1 << 20) && (page_size & (page_size - 1)) == 0,
          MSA_ERR_UNSUPPORTED, "page size %d (a power of two from %d to 2^20)", page_size, kMinPage);
  REQUIRE(n_pages >= 1 && (int64_t)n_pages * page_size < (1ll << 31), MSA_ERR_INVALID_ARG,
          "n_pages %d (the pool holds 1 to 2^31 - 1 rows)", n_pages);
  REQUIRE(max_pages >= 1 && (int64_t)max_pages * page_size <= (1ll << 30), MSA_ERR_INVALID_ARG,
          "max_pages %d (a request holds up to 2^30 rows)", max_pages);
  REQUIRE(n_req >= 0, MSA_ERR_INVALID_ARG, "n_req %d", n_req);
  REQUIRE(n_req <= msa::kPagedMaxReq, MSA_ERR_UNSUPPORTED, "n_req %d (up to %d)", n_req,
          msa::kPagedMaxReq);
  return MSA_OK;
}

msa_status check_heads(int32_t h_kv, int32_t d, int32_t dtype) {
  REQUIRE(dtype == MSA_FP32 || dtype == MSA_BF16, MSA_ERR_UNSUPPORTED, "dtype %d", dtype);
  REQUIRE(d == 64 || d == 128, MSA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", d);
  REQUIRE(h_kv >= 1, MSA_ERR_INVALID_ARG, "h_kv %d", h_kv);
  REQUIRE(h_kv <= kMaxHeads, MSA_ERR_UNSUPPORTED, "h_kv %d (up to %d)", h_kv, kMaxHeads);
  return MSA_OK;
}

// theta_i / (2 pi) mod 1 as 64-bit binary fractions, as msa::rope_turns, by repeated products
// instead of a power each: these calls are made per layer and token, and 64 extended-precision
// powers take 28 us of the host's time (0.6 us this way). The products' roundings add up to less
// than 2^-57 of theta_i: at positions below 2^31, 2^-28 of a turn.
void rope_fractions(double base, int d, unsigned long long* out) {
  const long double ratio = powl((long double)base, -2.0L / (long double)d);
  long double turns = 1.0L / 6.283185307179586476925286766559005768L;
  for (int i = 0; i < d / 2; ++i, turns *= ratio) {
    const long double scaled = (turns - floorl(turns)) * 18446744073709551616.0L;
    out[i] = scaled >= 18446744073709551615.0L ? ~0ull : (unsigned long long)scaled;
  }
}

}  // namespace

extern "C" {

size_t msa_page_plan_workspace(int32_t n_req, int32_t max_rows) {
  if (n_req < 0 || max_rows < 0) return kHeader;
  return kHeader + ((msa::page_plan_sums_bytes(n_req, max_rows) + 255) & ~(size_t)255);
}

msa_status msa_page_plan(const int32_t* target_len, const int32_t* len_in,
                         const int32_t* n_free_in, int32_t n_req, int32_t page_size,
                         int32_t max_pages, int32_t n_pages, int32_t max_rows,
                         int32_t* block_table, int32_t* free_list, int32_t* len_out,
                         int32_t* n_free_out, int32_t* row_start, int32_t* slot_map,
                         int32_t* row_pos, void* ws, size_t ws_bytes, void* stream) {
  msa_status s = check_pool(page_size, n_pages, max_pages, n_req);
  if (s != MSA_OK) return s;
  REQUIRE(max_rows >= 0, MSA_ERR_INVALID_ARG, "max_rows %d", max_rows);
  const size_t need = msa_page_plan_workspace(n_req, max_rows);
  REQUIRE(ws != nullptr && ws_bytes >= need && aligned(ws, 256), MSA_ERR_WORKSPACE,
          "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes, need);
  REQUIRE(n_free_in && n_free_out && row_start && free_list, MSA_ERR_INVALID_ARG, "null pointer");
  REQUIRE(n_req == 0 || (target_len && len_in && block_table && len_out), MSA_ERR_INVALID_ARG,
          "null pointer");
  REQUIRE(max_rows == 0 || (slot_map && row_pos), MSA_ERR_INVALID_ARG, "null row map");
  msa::PagePlanParams p{};
  p.target = target_len;
  p.len_in = len_in;
  p.nfree_in = n_free_in;
  p.table = block_table;
  p.free_list = free_list;
  p.len_out = len_out;
  p.nfree_out = n_free_out;
  p.row_start = row_start;
  p.slot_map = slot_map;
  p.row_pos = row_pos;
  p.n_req = n_req;
  p.max_pages = max_pages;
  p.n_pages = n_pages;
  p.page_shift = log2i(page_size);
  p.max_rows = max_rows;
  p.vec = aligned(slot_map, 16) && aligned(row_pos, 16);
  p.err = static_cast<int*>(ws);
  if (msa::page_plan_sums_bytes(n_req, max_rows) > 0)
    p.sums = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(ws) + kHeader);
  return done(msa::launch_page_plan(p, sm_count(), (cudaStream_t)stream), "msa_page_plan launch");
}

msa_status msa_paged_append_step(void* K_pages, void* V_pages, int32_t n_pages, int32_t page_size,
                                 const int32_t* slot_map, const int32_t* row_pos,
                                 const void* K_new, const void* V_new, int64_t k_stride,
                                 int64_t v_stride, int32_t n_rows, int32_t h_kv, int32_t d,
                                 int32_t dtype, int32_t pos0, float rope_base,
                                 const int32_t* planned, void* ws, size_t ws_bytes, void* stream) {
  msa_status s = check_heads(h_kv, d, dtype);
  if (s == MSA_OK) s = check_pool(page_size, n_pages, 1, 0);
  if (s != MSA_OK) return s;
  REQUIRE(n_rows >= 0 && pos0 >= 0, MSA_ERR_INVALID_ARG, "bad sizes (n_rows=%d pos0=%d)", n_rows,
          pos0);
  REQUIRE(ws != nullptr && ws_bytes >= kHeader && aligned(ws, 256), MSA_ERR_WORKSPACE,
          "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes, kHeader);
  if (n_rows == 0 && planned == nullptr) return done(cudaSuccess, "");
  const int64_t row = (int64_t)h_kv * d, per16 = 16 / (int64_t)esize(dtype);
  REQUIRE(n_rows == 0 || (slot_map && row_pos && K_new && V_new && K_pages && V_pages),
          MSA_ERR_INVALID_ARG, "null tensor");
  REQUIRE(k_stride >= row && v_stride >= row && k_stride % per16 == 0 && v_stride % per16 == 0,
          MSA_ERR_INVALID_ARG, "row strides %lld, %lld (at least h_kv * d, multiples of 16 bytes)",
          (long long)k_stride, (long long)v_stride);
  REQUIRE(aligned(K_new, 16) && aligned(V_new, 16) && aligned(K_pages, 16) && aligned(V_pages, 16),
          MSA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  msa::PagedAppendParams p{};
  p.K_new = K_new;
  p.V_new = V_new;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slot_map = slot_map;
  p.row_pos = row_pos;
  p.K_pages = K_pages;
  p.V_pages = V_pages;
  p.n_slots = n_pages * page_size;  // below 2^31
  p.n_rows = n_rows;
  p.planned = planned;
  p.h_kv = h_kv;
  p.pos0 = pos0;
  const bool rope = rope_base > 0.f;
  if (rope) rope_fractions((double)rope_base, d, p.rope_turns);
  p.err = static_cast<int*>(ws);
  return done(msa::launch_paged_append(p, rope, dtype, d, sm_count(), (cudaStream_t)stream),
              "msa_paged_append launch");
}

msa_status msa_paged_append(void* K_pages, void* V_pages, int32_t n_pages, int32_t page_size,
                            const int32_t* slot_map, const int32_t* row_pos, const void* K_new,
                            const void* V_new, int64_t k_stride, int64_t v_stride,
                            int32_t n_rows, int32_t h_kv, int32_t d, int32_t dtype, int32_t pos0,
                            float rope_base, void* ws, size_t ws_bytes, void* stream) {
  return msa_paged_append_step(K_pages, V_pages, n_pages, page_size, slot_map, row_pos, K_new,
                               V_new, k_stride, v_stride, n_rows, h_kv, d, dtype, pos0, rope_base,
                               nullptr, ws, ws_bytes, stream);
}

size_t msa_paged_attend_workspace(int32_t n_rows, int32_t n_req, int32_t h_q, int32_t h_kv,
                                  int32_t d, int32_t dtype, int32_t max_ctx, int32_t max_pages,
                                  int32_t page_size) {
  if (n_rows < 1 || n_req < 1 || h_kv < 1 || h_kv > kMaxHeads || h_q < h_kv || d < 1)
    return kHeader;
  (void)max_ctx;
  (void)max_pages;
  (void)page_size;
  return kHeader +
         msa::paged_attend_plan(n_rows, n_req, h_q, h_kv, d, dtype, sm_count()).bytes();
}

msa_status msa_paged_attend_step(const void* Q, int64_t q_stride, int32_t n_rows, int32_t h_q,
                                 const int32_t* row_start, const int32_t* len, int32_t n_req,
                                 const void* K_pages, const void* V_pages, int32_t n_pages,
                                 int32_t page_size, const int32_t* block_table, int32_t max_pages,
                                 const void* ctxK, const void* ctxV, const int32_t* ctx_len,
                                 int32_t max_ctx, int32_t h_kv, int32_t d, int32_t dtype,
                                 int32_t pos0, float rope_base, float scale, void* O, void* ws,
                                 size_t ws_bytes, void* step_ws, void* stream) {
  msa_status s = check_heads(h_kv, d, dtype);
  if (s == MSA_OK) s = check_pool(page_size, n_pages, max_pages, n_req);
  if (s != MSA_OK) return s;
  REQUIRE(h_q >= h_kv && h_q % h_kv == 0, MSA_ERR_INVALID_ARG, "h_q %d not a multiple of h_kv %d",
          h_q, h_kv);
  REQUIRE(h_q <= kMaxQueryHeads, MSA_ERR_UNSUPPORTED, "h_q %d (up to %d)", h_q, kMaxQueryHeads);
  REQUIRE(n_rows >= 0 && (int64_t)n_rows * h_q < (1ll << 31) && max_ctx >= 0 && pos0 >= 0,
          MSA_ERR_INVALID_ARG, "bad sizes (n_rows=%d h_q=%d max_ctx=%d pos0=%d)", n_rows, h_q,
          max_ctx, pos0);
  REQUIRE((int64_t)n_req * max_ctx < (1ll << 31), MSA_ERR_INVALID_ARG,
          "n_req * max_ctx %lld (below 2^31)", (long long)n_req * max_ctx);
  REQUIRE(scale == scale && std::fabs(scale) <= 3.0e38f, MSA_ERR_INVALID_ARG,
          "scale is not finite");
  const bool any = n_rows > 0 && n_req > 0;
  msa::PagedPlan pl{};
  if (any) pl = msa::paged_attend_plan(n_rows, n_req, h_q, h_kv, d, dtype, sm_count());
  const size_t need = kHeader + pl.bytes();
  REQUIRE(ws != nullptr && ws_bytes >= need && aligned(ws, 256), MSA_ERR_WORKSPACE,
          "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes, need);
  REQUIRE(aligned(step_ws, 256), MSA_ERR_WORKSPACE, "the step's workspace is not 256-byte aligned");
  const int64_t per16 = 16 / (int64_t)esize(dtype);
  if (any) {
    REQUIRE(Q && row_start && len && K_pages && V_pages && block_table && O, MSA_ERR_INVALID_ARG,
            "null tensor");
    REQUIRE(max_ctx == 0 || (ctxK && ctxV && ctx_len), MSA_ERR_INVALID_ARG, "null context");
    REQUIRE(q_stride >= (int64_t)h_q * d && q_stride % per16 == 0, MSA_ERR_INVALID_ARG,
            "Q row stride %lld (at least h_q * d, a multiple of 16 bytes)", (long long)q_stride);
    REQUIRE(aligned(Q, 16) && aligned(K_pages, 16) && aligned(V_pages, 16) && aligned(O, 16) &&
                (max_ctx == 0 || (aligned(ctxK, 16) && aligned(ctxV, 16))),
            MSA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (!any)  // nothing to do but to start the status word
    return done(cudaMemsetAsync(ws, 0, sizeof(int32_t), st), "msa_paged_attend");
  msa::PagedAttendParams p{};
  p.Q = Q;
  p.q_stride = q_stride;
  p.row_start = row_start;
  p.len = len;
  p.n_rows = n_rows;
  p.n_req = n_req;
  p.h_q = h_q;
  p.h_kv = h_kv;
  p.K_pages = K_pages;
  p.V_pages = V_pages;
  p.n_pages = n_pages;
  p.page_shift = log2i(page_size);
  p.table = block_table;
  p.max_pages = max_pages;
  p.cK = ctxK;
  p.cV = ctxV;
  p.ctx_len = max_ctx > 0 ? ctx_len : nullptr;
  p.max_ctx = max_ctx;
  p.rope = rope_base > 0.f ? 1 : 0;
  p.pos0 = pos0;
  if (p.rope) rope_fractions((double)rope_base, d, p.rope_turns);
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)d)) * 1.4426950408889634f;
  p.O = O;
  unsigned char* w8 = static_cast<unsigned char*>(ws);
  auto take = [&](size_t bytes) {
    unsigned char* at = w8;
    w8 += bytes;
    return at;
  };
  p.err = reinterpret_cast<int*>(take(kHeader));
  p.step_err = static_cast<int*>(step_ws);
  p.err_cta = reinterpret_cast<int*>(take(pl.err_bytes));
  p.tail = reinterpret_cast<int4*>(take(pl.tail_bytes));
  p.part_ml = reinterpret_cast<float*>(take(pl.ml_bytes));
  p.part_o = reinterpret_cast<float*>(take(pl.o_bytes));
  p.tc_tail = reinterpret_cast<int4*>(take(pl.tc_tail_bytes));
  p.tc_ml = reinterpret_cast<float*>(take(pl.tc_ml_bytes));
  p.tc_o = reinterpret_cast<float*>(take(pl.tc_o_bytes));
  p.q_rot = reinterpret_cast<__nv_bfloat16*>(take(pl.q_bytes));
  p.tc_rows = pl.tc_grid > 0 ? msa::kPagedWarpRows : INT32_MAX;
  p.tc_err_at = pl.grid;
  p.wait_limit = msa::device_wait_limit();
  return done(msa::launch_paged_attend(p, pl, dtype, d, st), "msa_paged_attend launch");
}

msa_status msa_paged_attend(const void* Q, int64_t q_stride, int32_t n_rows, int32_t h_q,
                            const int32_t* row_start, const int32_t* len, int32_t n_req,
                            const void* K_pages, const void* V_pages, int32_t n_pages,
                            int32_t page_size, const int32_t* block_table, int32_t max_pages,
                            const void* ctxK, const void* ctxV, const int32_t* ctx_len,
                            int32_t max_ctx, int32_t h_kv, int32_t d, int32_t dtype,
                            int32_t pos0, float rope_base, float scale, void* O, void* ws,
                            size_t ws_bytes, void* stream) {
  return msa_paged_attend_step(Q, q_stride, n_rows, h_q, row_start, len, n_req, K_pages, V_pages,
                               n_pages, page_size, block_table, max_pages, ctxK, ctxV, ctx_len,
                               max_ctx, h_kv, d, dtype, pos0, rope_base, scale, O, ws, ws_bytes,
                               nullptr, stream);
}

}  // extern "C"
