// paged.cu - the paged, ragged local context of sparse generation: the step's block tables and
// slot maps from the requests' lengths, and the append of the step's rows into their pages.
//
// Sparse generation keeps a request's local context next to its fixed routed memory
//   [news.neo-ai.one article, "推論パイプライン"; ruixiangma.github.io blog, "三阶段推理流程"];
// here the local contexts of many requests of different lengths share one pool of pages of
// 2^page_shift rows. Request r holds ceil(len_r / page) pages, listed in its row of the block
// table; pages nobody holds lie on a stack (free_list, its first n_free entries).
#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"
#include "paged.cuh"

namespace msa {
namespace pgd {

// ------------------------------------------------------------------------------ plan
// With old = len_in, tgt = target, held(x) = ceil(x / page): request r gives back the pages of its
// table columns [held(tgt), held(old)) or needs pages for the columns [held(old), held(tgt)).
// Three exclusive sums over the requests (new rows, needed pages, returned pages) fix everything
// else: the stack after the returns is free_list[0 .. F) followed by the returned pages in request
// order, and the i-th needed page is the i-th from its top, so with R returns it is returned page
// R-1-i, or free_list[F-1-(i-R)] for i >= R. Returned pages beyond the needed ones (R > P) stay on
// the stack at F .. F+R-P. No step depends on another's writes: entries read (below F; columns
// below held(old)) are never entries written, so one pass over the rows fills the slots and the
// table together. One CTA forms the sums and, for up to kPlanOneCta rows, fills the maps itself
// (one launch; a token for each of 256 requests: 6.1 us); more rows are filled by a second
// launch that is set up meanwhile (a cluster that did both was held up by its sixteen SMs'
// arithmetic: 14.6 us for 225,000 rows). One launch and two: 256 requests with 1,024 new rows 4.2
// and 6.1 us, 4,096 rows 5.2 and 6.4, 8,192 rows 7.2 and 7.3, 16,384 rows 11.2 and 7.0; 4,096
// requests of one row 12.1 and 15.8. Latency-bound.
constexpr int kPlanThreads = 1024;
constexpr int kPlanOneCta = 4096;  // rows up to which a single CTA fills the maps
constexpr int kFillThreads = 256;
constexpr int kAppendCtas = 8;     // CTAs of the append that an SM holds: its grid is one wave

// what the sums leave for the fill
struct PlanHead {
  int rows, F, P, R;
};
// the sums of every request, in shared memory or (for the second launch) in the workspace
struct PlanArrays {
  const int32_t* row;   // [n + 1] first new row of request r
  const int32_t* need;  // [n + 1] first needed page
  const int32_t* back;  // [n + 1] first returned page
  const int32_t* old;   // [n]
  const int32_t* tgt;   // [n]
};

struct PlanSums {
  long long rows, need, back;
};

// inclusive block scan of three values; totals of the block in *tot
__device__ __forceinline__ PlanSums block_scan(PlanSums v, PlanSums* warp_tot, PlanSums* tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, v.rows, o);
    const long long b = __shfl_up_sync(0xffffffffu, v.need, o);
    const long long c = __shfl_up_sync(0xffffffffu, v.back, o);
    if (lane >= o) {
      v.rows += a;
      v.need += b;
      v.back += c;
    }
  }
  if (lane == 31) warp_tot[warp] = v;
  __syncthreads();
  if (warp == 0) {
    PlanSums w = warp_tot[lane];
    const PlanSums own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, w.rows, o);
      const long long b = __shfl_up_sync(0xffffffffu, w.need, o);
      const long long c = __shfl_up_sync(0xffffffffu, w.back, o);
      if (lane >= o) {
        w.rows += a;
        w.need += b;
        w.back += c;
      }
    }
    if (lane == 31) *tot = w;
    warp_tot[lane] = PlanSums{w.rows - own.rows, w.need - own.need, w.back - own.back};
  }
  __syncthreads();
  const PlanSums base = warp_tot[warp];
  const PlanSums r{v.rows + base.rows, v.need + base.need, v.back + base.back};
  return r;
}

// last r in [0, n) with start[r] <= x (start non-decreasing, start[0] = 0): of requests
// without entries the last one, which is the one that owns entry x
__device__ __forceinline__ int owner(const int32_t* start, int n, int x) {
  int lo = 0, hi = n;  // start[lo] <= x, (hi == n or start[hi] > x)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The rows of threads gt of nt, four consecutive ones at a time: one search, then a walk along
// the requests.
__device__ __forceinline__ void plan_fill(const PagePlanParams& p, const PlanArrays& a,
                                          const PlanHead& h, int gt, int nt) {
  const int n = p.n_req, sh = p.page_shift, pm = (1 << sh) - 1;
  const int F = h.F, R = h.R;
  auto returned = [&](int q) {  // the q-th returned page
    const int r = owner(a.back, n, q);
    const int ht = (int)(((long long)a.tgt[r] + pm) >> sh);
    return p.table[(int64_t)r * p.max_pages + ht + (q - a.back[r])];
  };
  auto popped = [&](int i) {    // the i-th page off the stack
    return i < R ? returned(R - 1 - i) : p.free_list[F - 1 - (i - R)];
  };
  for (int q = gt; q < R - h.P; q += nt) p.free_list[F + q] = returned(q);
  bool bad_page = false;
#pragma unroll 1
  for (int64_t g = gt; g * 4 < p.max_rows; g += nt) {
    const int i0 = (int)g * 4;
    int32_t slot[4], pos[4];
    int r = i0 < h.rows ? owner(a.row, n, i0) : 0;
    int col = -1;
    int page = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e;
      slot[e] = pos[e] = -1;
      if (i >= h.rows) continue;
      while (a.row[r + 1] <= i) {
        ++r;
        col = -1;
      }
      const int at = a.old[r] + (i - a.row[r]);
      const int c = at >> sh;
      if (c != col) {
        col = c;
        const int ho = (int)(((long long)a.old[r] + pm) >> sh);
        page = c < ho ? p.table[(int64_t)r * p.max_pages + c] : popped(a.need[r] + (c - ho));
      }
      // the first row of a needed page enters it in the table
      if ((at & pm) == 0) p.table[(int64_t)r * p.max_pages + c] = page;
      pos[e] = at;
      const bool ok = page >= 0 && page < p.n_pages;
      bad_page |= !ok;
      slot[e] = ok ? (page << sh) + (at & pm) : -1;
    }
    if (p.vec && i0 + 3 < p.max_rows) {
      *reinterpret_cast<int4*>(p.slot_map + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.row_pos + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i0 + e < p.max_rows) {
          p.slot_map[i0 + e] = slot[e];
          p.row_pos[i0 + e] = pos[e];
        }
    }
  }
  if (bad_page) set_err(p.err, kErrBadIndex);
}

__global__ void __launch_bounds__(kPlanThreads, 1) page_plan_kernel(PagePlanParams p) {
  extern __shared__ int32_t sm[];
  const int n = p.n_req;
  int32_t* row_s = sm;                 // as PlanArrays
  int32_t* need_s = sm + (n + 1);
  int32_t* back_s = sm + 2 * (n + 1);
  int32_t* old_s = sm + 3 * (n + 1);
  int32_t* tgt_s = old_s + n;
  __shared__ PlanSums warp_tot[32], chunk_tot;
  __shared__ int bad_len;
  const int tid = threadIdx.x;
  const int sh = p.page_shift;
  const int pm = (1 << sh) - 1;
  const long long cap = (long long)p.max_pages << sh;
  wait_then_let_start();

  if (tid == 0) bad_len = 0;
  const int F = *p.nfree_in;
  PlanSums carry{0, 0, 0};
  __syncthreads();
  for (int b0 = 0; b0 < n; b0 += kPlanThreads) {
    const int r = b0 + tid;
    PlanSums v{0, 0, 0};
    int old = 0, tgt = 0;
    if (r < n) {
      old = p.len_in[r];
      tgt = p.target[r];
      if (old < 0 || tgt < 0 || old > cap || tgt > cap) {
        bad_len = 1;
        old = tgt = 0;
      }
      const int ho = (int)(((long long)old + pm) >> sh), ht = (int)(((long long)tgt + pm) >> sh);
      v.rows = max(tgt - old, 0);
      v.need = max(ht - ho, 0);
      v.back = max(ho - ht, 0);
    }
    const PlanSums s = block_scan(v, warp_tot, &chunk_tot);
    if (r < n) {  // sums past 2^31 are caught below, before they are used
      row_s[r] = (int32_t)(carry.rows + s.rows - v.rows);
      need_s[r] = (int32_t)(carry.need + s.need - v.need);
      back_s[r] = (int32_t)(carry.back + s.back - v.back);
      old_s[r] = old;
      tgt_s[r] = tgt;
    }
    carry.rows += chunk_tot.rows;
    carry.need += chunk_tot.need;
    carry.back += chunk_tot.back;
    __syncthreads();  // chunk_tot and warp_tot are reused
  }
  int code = 0;
  if (bad_len || F < 0 || F > p.n_pages || F + carry.back > p.n_pages) code = kErrBadIndex;
  else if (carry.need > F + carry.back || carry.rows > p.max_rows) code = kErrCtxOverflow;
  const PlanHead h{code ? 0 : (int)carry.rows, F, code ? 0 : (int)carry.need,
                   code ? 0 : (int)carry.back};
  if (tid == 0) {
    row_s[n] = (int32_t)carry.rows;
    need_s[n] = (int32_t)carry.need;
    back_s[n] = (int32_t)carry.back;
    *p.err = code;
    p.row_start[n] = h.rows;
    *p.nfree_out = F + h.R - h.P;  // (the count was read before the first barrier)
  }
  __syncthreads();
  for (int r = tid; r < n; r += kPlanThreads) {
    p.row_start[r] = code ? 0 : row_s[r];
    // a refused plan keeps the lengths; len_out may be len_in: every thread reads its own first
    p.len_out[r] = code ? p.len_in[r] : tgt_s[r];
  }
  if (p.sums == nullptr) {
    plan_fill(p, PlanArrays{row_s, need_s, back_s, old_s, tgt_s}, h, tid, kPlanThreads);
  } else {
    if (tid == 0) *reinterpret_cast<PlanHead*>(p.sums) = h;
    for (int i = tid; i < 5 * n + 3; i += kPlanThreads) p.sums[4 + i] = sm[i];
  }
}

__global__ void __launch_bounds__(kFillThreads) page_fill_kernel(PagePlanParams p) {
  wait_then_let_start();
  const PlanHead h = *reinterpret_cast<const PlanHead*>(p.sums);
  const int32_t* a = p.sums + 4;
  const int n = p.n_req;
  plan_fill(p, PlanArrays{a, a + (n + 1), a + 2 * (n + 1), a + 3 * (n + 1), a + 3 * (n + 1) + n},
            h, blockIdx.x * kFillThreads + threadIdx.x, gridDim.x * kFillThreads);
}

// ------------------------------------------------------------------------------ append
// K_pages[slot] = R(pos0 + pos) K_new, V_pages[slot] = V_new. A warp takes a row: lane = one
// 16-byte chunk of the lower half of a head and its partner half a head on (RoPE pairs
// i, i + d/2), so a row's angles are computed once and serve every head. HBM-bound for many
// rows (each row read and written once), latency for few.
template <typename T, int D, bool ROPE>
__global__ void __launch_bounds__(128, kAppendCtas) paged_append_kernel(PagedAppendParams p) {
  constexpr int E = 16 / sizeof(T);   // elements of a chunk
  constexpr int HC = D / 2 / E;       // chunks of half a head
  constexpr int HPW = 32 / HC;        // heads a warp takes at once
  using V = Vec<T, E>;
  using Raw = typename V::raw;
  const int lane = threadIdx.x & 31;
  const int c = lane % HC, h0 = lane / HC;
  unsigned long long F[E];
#pragma unroll
  for (int e = 0; e < E; ++e) F[e] = p.rope_turns[c * E + e];
  const int nw = gridDim.x * (blockDim.x >> 5);
  wait_then_let_start();
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.planned != nullptr && *p.planned > p.n_rows)
    set_err(p.err, kErrBadIndex);  // rows have a place and are not given
  for (int r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < p.n_rows; r += nw) {
    const int64_t slot = p.slot_map[r];
    if (slot < 0) continue;  // a padding row
    if (slot >= p.n_slots) {
      if (lane == 0) set_err(p.err, kErrBadIndex);
      continue;
    }
    const int64_t pos = (int64_t)p.pos0 + p.row_pos[r];
    const T* ks = static_cast<const T*>(p.K_new) + r * p.k_stride;
    const T* vs = static_cast<const T*>(p.V_new) + r * p.v_stride;
    T* kd = static_cast<T*>(p.K_pages) + slot * p.h_kv * D;
    T* vd = static_cast<T*>(p.V_pages) + slot * p.h_kv * D;
    float2 cs[E];
    if constexpr (ROPE) {
#pragma unroll
      for (int e = 0; e < E; ++e) cs[e] = rot_turns(pos, F[e]);
    }
    // two heads a turn, their loads in flight together
    for (int hh = h0; hh < p.h_kv; hh += 2 * HPW) {
      Raw ka[2], kb[2], va[2], vb[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int h = hh + u * HPW, at = h * D + c * E;
        if (h >= p.h_kv) continue;
        ka[u] = *reinterpret_cast<const Raw*>(ks + at);
        kb[u] = *reinterpret_cast<const Raw*>(ks + at + D / 2);
        va[u] = *reinterpret_cast<const Raw*>(vs + at);
        vb[u] = *reinterpret_cast<const Raw*>(vs + at + D / 2);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int h = hh + u * HPW, at = h * D + c * E;
        if (h >= p.h_kv) continue;
        Raw oa = ka[u], ob = kb[u];
        if constexpr (ROPE) {  // (turned by angle 0, an infinity's partner would be NaN)
          float a[E], b[E];
          V::unpack(ka[u], a);
          V::unpack(kb[u], b);
          T* ta = reinterpret_cast<T*>(&oa);
          T* tb = reinterpret_cast<T*>(&ob);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            ta[e] = Elem<T>::from_f(a[e] * cs[e].x - b[e] * cs[e].y);
            tb[e] = Elem<T>::from_f(b[e] * cs[e].x + a[e] * cs[e].y);
          }
        }
        *reinterpret_cast<Raw*>(kd + at) = oa;
        *reinterpret_cast<Raw*>(kd + at + D / 2) = ob;
        *reinterpret_cast<Raw*>(vd + at) = va[u];
        *reinterpret_cast<Raw*>(vd + at + D / 2) = vb[u];
      }
    }
  }
}

}  // namespace pgd

size_t page_plan_sums_bytes(int n_req, int max_rows) {
  return max_rows <= pgd::kPlanOneCta ? 0 : sizeof(int32_t) * (5 * (size_t)n_req + 3 + 4);
}

cudaError_t launch_page_plan(const PagePlanParams& p, int sms, cudaStream_t st) {
  const size_t smem = sizeof(int32_t) * (5 * (size_t)p.n_req + 3);
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = allow_smem_once(reinterpret_cast<const void*>(pgd::page_plan_kernel),
                                  sizeof(int32_t) * (5 * (size_t)kPagedMaxReq + 3), ready);
  if (e != cudaSuccess) return e;
  e = launch_early(pgd::page_plan_kernel, dim3(1), dim3(pgd::kPlanThreads), smem, st, p);
  if (e != cudaSuccess || p.sums == nullptr) return e;
  const int per = 4 * pgd::kFillThreads;
  const int grid = (int)std::min(((int64_t)p.max_rows + per - 1) / per, (int64_t)sms * 8);
  return launch_early(pgd::page_fill_kernel, dim3(grid), dim3(pgd::kFillThreads), 0, st, p);
}

cudaError_t launch_paged_append(const PagedAppendParams& p, bool rope, int dtype, int d, int sms,
                                cudaStream_t st) {
  const int grid = std::max(1, std::min((p.n_rows + 3) / 4, sms * pgd::kAppendCtas));
  auto go = [&](auto plain, auto turned) {
    return launch_early(rope ? turned : plain, dim3(grid), dim3(128), 0, st, p);
  };
  using pgd::paged_append_kernel;
  using bf16 = __nv_bfloat16;
  if (dtype == 1)
    return d == 128 ? go(paged_append_kernel<bf16, 128, false>, paged_append_kernel<bf16, 128, true>)
                    : go(paged_append_kernel<bf16, 64, false>, paged_append_kernel<bf16, 64, true>);
  return d == 128 ? go(paged_append_kernel<float, 128, false>, paged_append_kernel<float, 128, true>)
                  : go(paged_append_kernel<float, 64, false>, paged_append_kernel<float, 64, true>);
}

}  // namespace msa
