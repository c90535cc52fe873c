// paged.cuh - what the kernels of the paged attention share: a request's geometry on the device.
#pragma once

#include <climits>

#include "common.cuh"
#include "kernels.cuh"

namespace msa {

// The kernels before this one in the stream are complete; the next one may be set up. Until then
// this one may live beside kernels that write what it reads, so none of the paged kernels loads
// through the non-coherent path (read-only data of the kernel's whole life).
__device__ __forceinline__ void wait_then_let_start() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

struct PagedReq {
  int a, T, L, C;  // first row, new tokens, local rows, memory rows
};

// Request r if it has more than `lo` and at most `hi` query rows per KV head, else one without
// tokens. A length out of range and row starts that decrease or pass n_rows are recorded in
// *bad, and the request is left out (its rows of O are not written).
__device__ __forceinline__ PagedReq paged_req(const PagedAttendParams& p, int r, int lo, int hi,
                                              int* bad) {
  PagedReq q;
  q.a = p.row_start[r];
  q.T = p.row_start[r + 1] - q.a;
  q.L = p.len[r];
  q.C = p.ctx_len != nullptr ? min(max(p.ctx_len[r], 0), p.max_ctx) : 0;
  const bool ok = q.a >= 0 && q.T >= 0 && q.T <= p.n_rows - q.a && q.L >= 0 &&
                  q.L <= ((long long)p.max_pages << p.page_shift);
  if (!ok) *bad = kErrBadIndex;
  const int rows = ok ? q.T * (p.h_q / p.h_kv) : 0;  // n_rows * h_q is below 2^31
  if (!ok || rows <= lo || rows > hi) q.a = q.T = q.L = q.C = 0;
  return q;
}

}  // namespace msa
