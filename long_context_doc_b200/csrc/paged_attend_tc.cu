// paged_attend_tc.cu - the paged attention of paged_attend.cu for requests with more than a
// handful of query rows per KV head (chunks of a prompt, drafted tokens) on the 5th-generation
// tensor cores; bf16. The operation, its masks and its refusals are those of that file.
//
// One persistent CTA per SM over an equal share of the flattened list (request, KV head, block
// of up to 256 query rows, tile of 128 keys); a block that a share does not hold whole leaves a
// partial for the merge kernel. A block is two halves of 128 rows (TMEM lanes), each with its
// own scores and accumulator in TMEM, worked on in alternation: while one half's softmax runs,
// the tensor cores form the other half's products, and both halves use every K and V tile that
// was loaded. Warp 0 copies the tiles (one TMA box of 64 dims per page and half a head) into a
// ring of K and V tiles; one thread of warp 1 issues tcgen05.mma: S = Q K^T, then O += P V with P
// read from TMEM, where the softmax put it over the scores, and V as an MN-major operand as
// stored. Warps 2-9 hold one query row per thread: they rotate and stage their half's queries,
// load the 128 scores of a tile from TMEM once, mask, and keep the running maximum (raised, with
// O rescaled in TMEM, only when a tile's maximum passes it by more than 8 in log2 units) and sum
// in fp32. A half's completed scores imply its earlier products (the issuing thread's MMAs
// complete in order), so O is rescaled and Q replaced without further waits.
// Every wait is bounded; on expiry the CTA records kErrWaitTimeout, lets its copies and MMAs
// land, frees its TMEM and leaves the rest unwritten.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"
#include "paged.cuh"

namespace msa {
namespace pgt {

constexpr int kN = 128;                   // keys of a tile
constexpr int kHalf = 128;                // query rows of a half
constexpr int kThreads = 320;
constexpr uint32_t kSlice = 128 * 128;    // 128 rows x 64 bf16, 128-byte swizzle: 16 KB
constexpr float kRaise = 8.f;

template <int D> struct Cfg {
  static constexpr int SL = D / 64;                    // slices of a tile
  static constexpr uint32_t kTile = SL * kSlice;       // K or V tile, and one half's Q
  static constexpr int NS = D == 128 ? 5 : 8;          // ring tiles
  static constexpr size_t smem = 1024 + 2 * kTile + NS * kTile + 512;
};

__device__ __forceinline__ void tma3(void* dst, const CUtensorMap* map, int x, int y, int z,
                                     uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// K-major operand slice [128 rows][64 bf16], 128-byte swizzle: 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t desc_k(const void* slice) {
  const uint64_t a = (uint64_t)(smem_u32(slice) & 0x3FFFFu) >> 4;
  return a | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// the same slices read along N: 64 elements of a row, the next 64 one slice on
__device__ __forceinline__ uint64_t desc_mn(const void* rows) {
  const uint64_t a = (uint64_t)(smem_u32(rows) & 0x3FFFFu) >> 4;
  return a | ((uint64_t)(kSlice >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {  // max relative error 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t par, int* err,
                                              volatile int* abort_flag) {
  if (mbar_try_wait(bar, par)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, par)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > kDefaultWaitLimit) {
      set_err(err, kErrWaitTimeout);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// ------------------------------------------------------------------ the list of work
// Geometry shared by all roles: blocks of TB = 256 / Gq tokens (rows t * Gq + head of the
// group); a block's tiles are the memory's and the local ones up to its last token's row.
struct Work {
  PagedReq q;
  int r, head, blk, nb, CT;
  int t0, t1;        // this CTA's tiles of the block, of n_tiles
  int n_tiles;
  int rows;          // query rows of the block
};
struct Walk {
  const PagedAttendParams& p;
  int Gq, TB;
  int64_t left;      // tiles of the share still to hand out
  __device__ __forceinline__ int blocks(const PagedReq& q) const { return (q.T + TB - 1) / TB; }
  __device__ __forceinline__ int tiles(const PagedReq& q, int blk) const {
    const int last = q.L - q.T + min(q.T, (blk + 1) * TB);  // rows the last token sees
    return max(1, (q.C + kN - 1) / kN + (max(last, 0) + kN - 1) / kN);
  }
  __device__ __forceinline__ int64_t request_tiles(const PagedReq& q) const {  // of one KV head
    int64_t n = 0;
    for (int b = 0, nb = blocks(q); b < nb; ++b) n += tiles(q, b);
    return n;
  }
  __device__ __forceinline__ void set(Work& w, int from) {
    w.n_tiles = tiles(w.q, w.blk);
    w.rows = min(TB, w.q.T - w.blk * TB) * Gq;
    w.t0 = from;
    w.t1 = (int)min((int64_t)w.n_tiles, from + left);
    left -= w.t1 - from;
  }
  __device__ __forceinline__ void enter(Work& w, int r) {
    int ignore = 0;
    w.r = r;
    w.q = paged_req(p, r, p.tc_rows, INT_MAX, &ignore);
    w.nb = blocks(w.q);
    w.CT = (w.q.C + kN - 1) / kN;
  }
  // The first block of a share that starts `off` tiles into request r's.
  __device__ __forceinline__ void first(Work& w, int r, int64_t off) {
    enter(w, r);
    const int64_t per_head = request_tiles(w.q);
    w.head = (int)(off / per_head);
    int64_t rem = off % per_head;
    for (w.blk = 0; rem >= tiles(w.q, w.blk); ++w.blk) rem -= tiles(w.q, w.blk);
    set(w, (int)rem);
  }
  // The next block (whole warps; called only while left > 0, so there is one).
  __device__ __forceinline__ void next(Work& w, int lane) {
    if (++w.blk == w.nb) {
      w.blk = 0;
      if (++w.head == p.h_kv) {
        w.head = 0;
        for (int r = w.r + 1;; r += 32) {  // requests without work are passed 32 at a time
          int ignore = 0;
          const int mine = r + lane;
          const bool has =
              mine < p.n_req && paged_req(p, mine, p.tc_rows, INT_MAX, &ignore).T > 0;
          const unsigned m = __ballot_sync(0xffffffffu, has);
          if (m || r + 32 > p.n_req) {
            enter(w, m ? r + __ffs(m) - 1 : w.r);
            break;
          }
        }
      }
    }
    set(w, 0);
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_attend_tc_kernel(const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ CUtensorMap map_ck,
                       const __grid_constant__ CUtensorMap map_cv,
                       const __grid_constant__ PagedAttendParams p) {
  using C = Cfg<D>;
  constexpr int NS = C::NS, KS = D / 16, SL = C::SL;
  extern __shared__ __align__(1024) unsigned char sm_raw[];
  unsigned char* base = smem_align1024(sm_raw);
  unsigned char* q_s = base;                       // [2 halves][SL][128][64]
  unsigned char* ring = base + 2 * C::kTile;       // [NS][SL][128][64]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + NS * C::kTile);
  uint64_t* full = bars;            // [NS] ring tile landed
  uint64_t* empty = bars + NS;      // [NS] ring tile consumed
  uint64_t* qfull = bars + 2 * NS;  // [2] a half's queries staged (128 threads)
  uint64_t* sfull = qfull + 2;      // [2] a half's scores written
  uint64_t* pfull = qfull + 4;      // [2] a half's probabilities written (128 threads)
  uint64_t* odone = qfull + 6;      // [2] a block's last P V of the half completed
  uint64_t* done = qfull + 8;       // every issued MMA completed
  __shared__ int64_t warp_tot[kThreads / 32];
  __shared__ int64_t start_off;
  __shared__ int start_r, cta_err;
  __shared__ int abort_word;
  __shared__ uint32_t tmem_holder;
  volatile int* abort_flag = &abort_word;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Gq = p.h_q / p.h_kv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&qfull[h], kHalf);
      mbar_init(&sfull[h], 1);
      mbar_init(&pfull[h], kHalf);
      mbar_init(&odone[h], 1);
    }
    mbar_init(done, 1);
    abort_word = 0;
    cta_err = 0;
    start_r = -1;
    fence_mbar_init();
  }
  __syncthreads();

  // the CTA's share of the list: total tiles first, then the request that holds the share's start
  Walk walk{p, Gq, 2 * kHalf / Gq, 0};
  int err = 0;
  int64_t total = 0, mine = 0;
  int G = 1;  // shares: no more than tiles, so that none of them is empty
  for (int pass = 0; pass < 2; ++pass) {
    const int64_t x0 = pass ? total * blockIdx.x / G : 0;
    int64_t carry = 0;
    for (int r0 = 0; r0 < p.n_req; r0 += kThreads) {
      const int r = r0 + tid;
      int64_t v = mine;
      if (pass == 0 || p.n_req > kThreads) {
        v = 0;
        if (r < p.n_req)
          v = walk.request_tiles(paged_req(p, r, p.tc_rows, INT_MAX, &err)) * p.h_kv;
        mine = v;
      }
      int64_t inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) warp_tot[warp] = inc;
      __syncthreads();
      int64_t before = carry;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_tot[w];
        carry += warp_tot[w];
      }
      const int64_t lo = before + inc - v;
      if (pass == 1 && v > 0 && lo <= x0 && x0 < lo + v) {
        start_r = r;
        start_off = x0 - lo;
      }
      __syncthreads();
    }
    total = carry;
    G = (int)min((int64_t)gridDim.x, total);
    if ((int)blockIdx.x >= G) break;
  }
  const bool work = (int)blockIdx.x < G;   // then start_r is set
  const int64_t x0 = work ? total * blockIdx.x / G : 0;
  const int64_t x1 = work ? total * (blockIdx.x + 1) / G : 0;
  walk.left = x1 - x0;
  int4 tail = make_int4(-1, 0, 0, 0);
  int tail_head = 0;

  if (work) {
    if (warp == 0) {  // scores of the halves at columns 0 and 128, accumulators at 256 and 384
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&tmem_holder)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_holder;
    Work w;
    walk.first(w, start_r, start_off);

    if (warp == 0) {
      // ---------------- copies: K then V of each tile, one page (or memory tile) a lane
      uint32_t seq = 0;
      const int ps = 1 << p.page_shift;
      const int br = min(ps, kN);               // rows of a box
      const int half = lane % SL, piece = lane / SL;
      bool ok = true;
      while (ok) {
        for (int t = w.t0; ok && t < w.t1; ++t) {
          const bool ctx = t < w.CT;
          const int k0 = (ctx ? t : t - w.CT) * kN;
          int row = 0;
          bool load;
          int rows_per = kN;
          if (ctx) {
            load = piece == 0;
            row = w.r * p.max_ctx + k0;
          } else {
            rows_per = br;
            const int k = k0 + piece * br;
            load = piece < kN / br && k < w.q.L;
            if (load) {
              const int page = __ldg(p.table + (int64_t)w.r * p.max_pages + (k >> p.page_shift));
              if (page < 0 || page >= p.n_pages) {
                err = kErrBadIndex;
                load = false;
              } else {
                row = (page << p.page_shift) + (k & (ps - 1));
              }
            }
          }
          const uint32_t bytes =
              __popc(__ballot_sync(0xffffffffu, load)) * (uint32_t)rows_per * 128u;
          for (int kv = 0; kv < 2; ++kv, ++seq) {
            const int s = seq % NS;
            if (seq >= NS) {
              ok = wait_or_abort(&empty[s], ((seq / NS) - 1) & 1, &cta_err, abort_flag);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
            __syncwarp();
            if (load) {
              const CUtensorMap* m = ctx ? (kv ? &map_cv : &map_ck) : (kv ? &map_v : &map_k);
              tma3(ring + s * C::kTile + half * kSlice + piece * br * 128, m, half * 64, w.head,
                   row, &full[s]);
            }
          }
        }
        if (walk.left == 0) break;
        walk.next(w, lane);
      }
      // the copies issued land before the CTA can exit
      for (uint32_t q = seq > NS ? seq - NS : 0; q < seq; ++q)
        mbar_wait_bounded(&full[q % NS], (q / NS) & 1, &cta_err);
    } else if (warp == 1) {
      // ---------------- MMA issuer
      constexpr uint32_t idesc_s = (1u << 4) | (1u << 7) | (1u << 10) |
                                   ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(kHalf >> 4) << 24);
      constexpr uint32_t idesc_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                   ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kHalf >> 4) << 24);
      uint32_t seq = 0;              // next ring tile
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
      auto wait = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, par, &cta_err, abort_flag));
      };
      auto wait_ring = [&](uint32_t q) { return wait(&full[q % NS], (q / NS) & 1); };
      auto scores = [&](int h, uint32_t q) {  // S_h = Q_h K^T
        fence_after();
        if (lane == 0) {
          const unsigned char* k = ring + (q % NS) * C::kTile;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk)
            mma_ss(tmem + h * 128, desc_k(q_s + h * C::kTile + (kk >> 2) * kSlice) + 2 * (kk & 3),
                   desc_k(k + (kk >> 2) * kSlice) + 2 * (kk & 3), idesc_s, kk ? 1u : 0u);
          commit(&sfull[h]);
        }
        __syncwarp();
      };
      auto product = [&](int h, uint32_t q, bool first) {  // O_h (+)= P_h V
        fence_after();
        if (lane == 0) {
          const unsigned char* v = ring + (q % NS) * C::kTile;
#pragma unroll
          for (int kk = 0; kk < kN / 16; ++kk)
            mma_ts(tmem + 256 + h * 128, tmem + h * 128 + kk * 8, desc_mn(v + kk * 2048), idesc_o,
                   (first && kk == 0) ? 0u : 1u);
        }
        __syncwarp();
      };
      auto release = [&](uint32_t q) {
        if (lane == 0) commit(&empty[q % NS]);
        __syncwarp();
      };
      bool ok = true;
      while (ok) {
        const int nh = w.rows > kHalf ? 2 : 1;
        const int n = w.t1 - w.t0;
        ok = wait_ring(seq);
        for (int h = 0; ok && h < nh; ++h) {
          ok = wait(&qfull[h], nq[h] & 1);
          ++nq[h];
          if (ok) scores(h, seq);
        }
        if (!ok) break;
        release(seq);
        ++seq;
        for (int j = 0; ok && j < n; ++j) {
          const bool last = j + 1 == n;
          for (int h = 0; ok && h < nh; ++h) {
            ok = wait(&pfull[h], np[h] & 1);
            ++np[h];
            if (ok && h == 0) ok = wait_ring(seq);
            if (!ok) break;
            product(h, seq, j == 0);
            if (h == nh - 1) release(seq);
            if (last) {
              if (lane == 0) commit(&odone[h]);
              __syncwarp();
            } else {
              if (h == 0) ok = wait_ring(seq + 1);
              if (!ok) break;
              scores(h, seq + 1);
              if (h == nh - 1) release(seq + 1);
            }
          }
          seq += last ? 1 : 2;
        }
        if (!ok || walk.left == 0) break;
        walk.next(w, lane);
      }
      if (lane == 0) commit(done);
      __syncwarp();
      mbar_wait_bounded(done, 0, &cta_err);
    } else {
      // ---------------- softmax: a half's 128 rows, one a thread
      const int h = (warp - 2) >> 2;
      const int lrow = (warp & 3) * 32 + lane;        // row in the half = TMEM lane
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_col = lane_base + h * 128, o_col = lane_base + 256 + h * 128;
      const float c = p.scale_log2;
      uint32_t nt = 0, nblk = 0;   // tiles and blocks this half has taken
      uint32_t seq = 0;            // ring tile of the block's first K
      auto wait = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, par, &cta_err, abort_flag));
      };
      // The warp's 32 query rows, rotated, rounded to bf16 and staged as the K-major operand.
      // A lane takes the RoPE pairs 2l, 2l + 1 of a row (D = 64: of one of two rows), so a
      // token's angles are computed once for the rows of its heads that follow one another.
      auto stage_q = [&](const Work& b) {
        constexpr int LPR = D / 4;             // lanes a row takes
        constexpr int RPS = 32 / LPR;          // rows at once
        const int l = lane % LPR;
        const int64_t pos0 = (int64_t)p.pos0 + b.q.L - b.q.T;
        const unsigned long long F0 = p.rope_turns[2 * l], F1 = p.rope_turns[2 * l + 1];
        int last_tok = -1;
        float2 c0 = make_float2(1.f, 0.f), c1 = c0;
#pragma unroll 4
        for (int i = 0; i < 32; i += RPS) {
          const int rr = (warp & 3) * 32 + i + lane / LPR;   // row in the half
          const int row = h * kHalf + rr;
          if (row < b.rows) {
            const int tok = b.blk * walk.TB + row / Gq;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.Q) +
                                       (int64_t)(b.q.a + tok) * p.q_stride +
                                       (b.head * Gq + row % Gq) * D;
            const uint32_t lo = __ldg(reinterpret_cast<const uint32_t*>(src) + l);
            const uint32_t hi = __ldg(reinterpret_cast<const uint32_t*>(src + D / 2) + l);
            if (p.rope && tok != last_tok) {
              last_tok = tok;
              c0 = rot_turns(pos0 + tok, F0);
              c1 = rot_turns(pos0 + tok, F1);
            }
            const float a0 = __uint_as_float(lo << 16), a1 = __uint_as_float(lo & 0xFFFF0000u);
            const float b0 = __uint_as_float(hi << 16), b1 = __uint_as_float(hi & 0xFFFF0000u);
            const uint32_t ra = pack_bf16(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
            const uint32_t rb = pack_bf16(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
            unsigned char* dst = q_s + h * C::kTile + rr * 128;
            // element e of the row: slice e / 64, 16-byte chunk (e % 64) / 8 ^ (row & 7)
            const int ea = 2 * l, eb = 2 * l + D / 2;
            *reinterpret_cast<uint32_t*>(dst + (ea >> 6) * kSlice +
                                         ((((ea & 63) >> 3) ^ (rr & 7)) << 4) + (ea & 7) * 2) = ra;
            *reinterpret_cast<uint32_t*>(dst + (eb >> 6) * kSlice +
                                         ((((eb & 63) >> 3) ^ (rr & 7)) << 4) + (eb & 7) * 2) = rb;
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&qfull[h]);
      };
      bool ok = true;
      if (h == 0 || w.rows > kHalf) stage_q(w);
      while (ok) {
        const bool active = h == 0 || w.rows > kHalf;
        const int n = w.t1 - w.t0;
        const bool begins = w.t0 == 0, ends = w.t1 == w.n_tiles;
        const Work b = w;
        const bool more = walk.left > 0;
        float m = -INFINITY, l0 = 0.f, l1 = 0.f;
        if (active) {
          const int row = h * kHalf + lrow;
          const bool any_row = h * kHalf + (warp & 3) * 32 < b.rows;  // of the warp
          const int tok = b.blk * walk.TB + min(row, b.rows - 1) / Gq;
          const int vis = b.q.L - b.q.T + tok;                        // last visible local row
          const int vis_first = b.q.L - b.q.T + b.blk * walk.TB + h * kHalf / Gq;
          for (int t = b.t0; t < b.t1; ++t, ++nt) {
            const bool ctx = t < b.CT;
            const int k0 = (ctx ? t : t - b.CT) * kN;
            const int valid = (ctx ? b.q.C : b.q.L) - k0;            // rows the tile holds
            ok = wait(&sfull[h], nt & 1);
            if (!ok) break;
            fence_after();
            if (any_row) {
              uint32_t sr[128];
#pragma unroll
              for (int i = 0; i < 4; ++i) ld32(s_col + i * 32, sr + i * 32);
              wait_ld();
              if (!(ctx ? valid >= kN : k0 + kN - 1 <= min(vis_first, b.q.L - 1))) {
                const int lim = min(valid - 1, ctx ? kN : vis - k0);  // keys [0, lim] visible
#pragma unroll
                for (int i = 0; i < 128; ++i)
                  if (i > lim) sr[i] = 0xFF800000u;                  // -inf
              }
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int i = 0; i < 128; i += 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(sr[i + e]));
              }
              const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
              const bool raise = mt > m + kRaise || (m == -INFINITY && mt != -INFINITY);
              if (__any_sync(0xffffffffu, raise)) {
                const float mn = raise ? mt : m;
                const float alpha = (raise && m != -INFINITY) ? ex2(m - mn) : 1.f;
                m = mn;
                l0 *= alpha;
                l1 *= alpha;
                if (t > b.t0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                  for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t ov[32];
                    ld32(o_col + ch * 32, ov);
                    wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                      ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                    st32(o_col + ch * 32, ov);
                  }
                }
              }
              // the probabilities in bf16 over the scores' columns (their sum in fp32)
              const float neg = m == -INFINITY ? 0.f : -m;
#pragma unroll
              for (int ch = 0; ch < 2; ++ch) {
                uint32_t pk[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float p0 = ex2(fmaf(__uint_as_float(sr[ch * 64 + 2 * i]), c, neg));
                  const float p1 = ex2(fmaf(__uint_as_float(sr[ch * 64 + 2 * i + 1]), c, neg));
                  l0 += p0;
                  l1 += p1;
                  pk[i] = pack_bf16(p0, p1);
                }
                st32(s_col + ch * 32, pk);
              }
              wait_st();
            }
            // V rows past the end hold anything: cleared, for 0 * NaN would reach O
            if (h == 0 && valid < kN) {
              const uint32_t q = seq + 2 * (t - b.t0) + 1;
              ok = wait(&full[q % NS], (q / NS) & 1);
              if (!ok) break;
              if (lrow >= valid) {
#pragma unroll
                for (int sl = 0; sl < SL; ++sl) {
                  uint4* vr = reinterpret_cast<uint4*>(ring + (q % NS) * C::kTile + sl * kSlice +
                                                       lrow * 128);
#pragma unroll
                  for (int i = 0; i < 8; ++i) vr[i] = make_uint4(0u, 0u, 0u, 0u);
                }
              }
              fence_proxy_async_smem();
            }
            fence_before();
            mbar_arrive(&pfull[h]);
          }
        }
        seq += 2 * n;
        if (!ok) break;
        // the next block's queries go out while this block's last product runs
        if (more) {
          walk.next(w, lane);
          if (h == 0 || w.rows > kHalf) stage_q(w);
        }
        if (active) {
          ok = wait(&odone[h], nblk & 1);
          ++nblk;
          if (!ok) break;
          fence_after();
          const int row = h * kHalf + lrow;
          const float l = l0 + l1;
          const bool whole = begins && ends;
          const float inv = l > 0.f ? 1.f / l : 0.f;
          const int tok = b.blk * walk.TB + row / Gq;
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.O) +
                               ((int64_t)(b.q.a + tok) * p.h_q + b.head * Gq + row % Gq) * D;
          const int64_t slot = ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * (2 * kHalf) + row;
          float* part = p.tc_o + slot * D;
          if (h * kHalf + (warp & 3) * 32 < b.rows) {
#pragma unroll
            for (int ch = 0; ch < D / 32; ++ch) {
              uint32_t ov[32];
              ld32(o_col + ch * 32, ov);
              wait_ld();
              if (row < b.rows) {
                if (whole) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    uint32_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      v[e] = pack_bf16(__uint_as_float(ov[8 * i + 2 * e]) * inv,
                                       __uint_as_float(ov[8 * i + 2 * e + 1]) * inv);
                    *reinterpret_cast<uint4*>(out + ch * 32 + 8 * i) =
                        make_uint4(v[0], v[1], v[2], v[3]);
                  }
                } else {
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(part + ch * 32 + 4 * i) =
                        make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
                }
              }
            }
            if (!whole && row < b.rows)
              *reinterpret_cast<float2*>(p.tc_ml + slot * 2) = make_float2(m, l);
          }
          fence_before();  // O is read before the next block's products
        }
        if (begins && !ends) {  // goes on in the next CTAs' shares
          const int64_t end = x1 - b.t1 + b.n_tiles - 1;
          tail = make_int4(b.q.a, b.q.T, b.blk,
                           (int)(((end + 1) * G + total - 1) / total - 1));
          tail_head = b.head;
        }
        if (!more) break;
      }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                   : "memory");
  }
  if (err) atomicCAS(&cta_err, 0, err);
  __syncthreads();
  if (tid == 64) {  // the first softmax thread knows the share's last block
    if (cta_err == kErrWaitTimeout) tail.x = -1;
    p.tc_tail[2 * blockIdx.x] = tail;
    p.tc_tail[2 * blockIdx.x + 1] = make_int4(tail_head, 0, 0, 0);
    p.err_cta[p.tc_err_at + blockIdx.x] = cta_err;
  }
  // the merge kernel waits for this grid only; this grid's end must include the end of the one
  // launched before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D>
cudaError_t launch(const PagedAttendParams& p, int grid, cudaStream_t st) {
  CUtensorMap mk, mv, mck, mcv;
  const uint64_t row = (uint64_t)D * 2;
  const uint64_t str[2] = {row, row * p.h_kv};
  {
    const uint64_t dims[3] = {D, (uint64_t)p.h_kv, (uint64_t)p.n_pages << p.page_shift};
    const uint32_t box[3] = {64, 1, (uint32_t)std::min(1 << p.page_shift, kN)};
    if (!encode_bf16_map(&mk, p.K_pages, 3, dims, str, box, true) ||
        !encode_bf16_map(&mv, p.V_pages, 3, dims, str, box, true))
      return cudaErrorInvalidValue;
  }
  if (p.max_ctx > 0) {
    const uint64_t dims[3] = {D, (uint64_t)p.h_kv, (uint64_t)p.n_req * p.max_ctx};
    const uint32_t box[3] = {64, 1, kN};
    if (!encode_bf16_map(&mck, p.cK, 3, dims, str, box, true) ||
        !encode_bf16_map(&mcv, p.cV, 3, dims, str, box, true))
      return cudaErrorInvalidValue;
  } else {  // no memory tiles: never read
    mck = mk;
    mcv = mv;
  }
  auto kfn = paged_attend_tc_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Cfg<D>::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, mk, mv, mck, mcv, p);
}

}  // namespace pgt

cudaError_t launch_paged_attend_tc(const PagedAttendParams& p, int grid, int d, cudaStream_t st) {
  return d == 128 ? pgt::launch<128>(p, grid, st) : pgt::launch<64>(p, grid, st);
}

}  // namespace msa
