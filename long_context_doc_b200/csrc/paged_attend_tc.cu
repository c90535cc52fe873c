// paged_attend_tc.cu - the paged attention of paged_attend.cu for requests with more than a
// handful of query rows per KV head (chunks of a prompt, drafted tokens) on the 5th-generation
// tensor cores; bf16. The operation, its masks and its refusals are those of that file.
//
// One persistent CTA per SM over an equal share of the flattened list (request, KV head, block
// of up to 256 query rows, tile of 128 keys); a block that a share does not hold whole leaves a
// partial for the merge kernel. A block is two halves of 128 rows (TMEM lanes), each with its
// own scores and accumulator in TMEM, worked on in alternation: while one half's softmax runs,
// the tensor cores form the other half's products, and both halves use every K and V tile that
// was loaded. Warp 0 walks the share, announces its blocks to the others and copies the tiles (one
// TMA box of 64 dims per page and half a head) into a ring, and a block's queries, which the
// warp-level kernel has rotated, rounded to bf16 and laid out as the operand wants them. Warp 1
// issues tcgen05.mma: S = Q K^T, then O += P V with P read from TMEM, where the softmax put it
// over the scores, and V as an MN-major operand as stored. Warps 2-9 hold one query row per
// thread: they load the 128 scores of a tile from TMEM once, mask, and keep the running maximum
// (raised, with O rescaled in TMEM, only when a tile's maximum passes it by more than 8 in log2
// units) and sum in fp32, and hand over the probabilities half a tile at a time. With two halves a
// half's completed scores imply its earlier products (the issuing thread's MMAs complete in
// order), so O is rescaled without further waits. A block of one half has both scores buffers to
// itself: the scores of a tile are formed before the product of the tile before it, and with the
// queries' low parts too (their place in shared memory is the other half's).
// Roundings: the probabilities to bf16 once, the queries of two halves as well (the mean error is
// 1.7 times that of the output's own rounding; one half: 1.4 times). For a chunk of 2,048 tokens
// over 32,768 rows the probabilities' low parts add 27%, the queries' of two halves 22% (a ring of
// three tiles instead of four, no staging of the output, half as many products again: 1.20 ms for
// 0.98, 1.33-1.51 for 1.09 at the power cap; 24 mixed requests 460-490 us for 380-420).
// Bound by the chain scores -> softmax -> product: tensor pipe and exponentials are each busy half
// of the time (2,048 tokens over 32,768 rows: 0.95-0.99 ms, 1.08-1.13 PFLOP/s, and 1.09-1.12 ms,
// 0.95-0.98 PFLOP/s, where replays back to back meet the power cap).
// Every wait is bounded (the softmax warps' for scores by the limit that
// msa_set_device_wait_limit sets); on expiry the CTA records kErrWaitTimeout, lets its copies and
// MMAs land, frees its TMEM and leaves the rest unwritten.
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
constexpr uint32_t kBounce = 32 * 128;    // a warp's 128 bytes of 32 rows on their way to memory
constexpr int kQueue = 4;                 // blocks announced ahead
constexpr float kRaise = 8.f;

template <int D> struct Cfg {
  static constexpr int SL = D / 64;                    // slices of a tile
  static constexpr uint32_t kTile = SL * kSlice;       // K or V tile, and one half's Q
  static constexpr int NS = D == 128 ? 4 : 8;          // ring tiles (5 measured the same)
  static constexpr size_t smem = 1024 + 2 * kTile + NS * kTile + 8 * kBounce + 512;
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
// The MMAs and commits are issued by one elected thread of a converged warp (always the same
// one), so that their operands are computed in uniform registers: issued under a branch on the
// lane, each operand's move into a uniform register made a 128 x 128 x 16 step take 137 clocks
// instead of the tensor cores' 64.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_u32(bar))
      : "memory");
}
// a value that every lane of the warp holds, as one the compiler knows to be so
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
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
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
// Bounded wait: gives up after the default limit (a second or so), or when another role has given
// up. The blocking form: warps that spun on the non-blocking test took issue slots from the other
// half's softmax (4% of a long chunk's time).
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t par, int* err,
                                              volatile int* abort_flag) {
  if (mbar_try_wait(bar, par)) return true;
  const long long t0 = clock64();
#pragma unroll 1
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

// The same with the limit of the call, which msa_set_device_wait_limit sets: polling, so that the
// limit and not the hardware's suspend time decides.
__device__ __forceinline__ bool poll_or_abort(uint64_t* bar, uint32_t par, long long limit, int* err,
                                              volatile int* abort_flag) {
  const long long t0 = clock64();
#pragma unroll 1
  while (!mbar_test_wait(bar, par)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > limit) {
      set_err(err, kErrWaitTimeout);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// ------------------------------------------------------------------ the list of work
// Blocks of TB = 256 / Gq tokens (rows t * Gq + head of the group); a block's tiles are the memory's
// and the local ones up to its last token's row. The list counts a unit for each tile (of one half
// or two: both take as long as their chain of products and softmax) and kStart before a block's
// first one. A tile belongs to the share that holds its unit. (24 mixed requests: 356 us with
// kStart = 0, 345 with 1, 342 with 2 and 3, 346 with 4; half a unit for a tile of one half: 365.)
constexpr int kStart = 2;
struct Work {
  PagedReq q;
  int r, head, blk, nb, CT;
  int t0, t1;        // this CTA's tiles of the block, of n_tiles
  int n_tiles;
  int toks, rows;    // tokens and query rows of the block
  int first;         // local row of its first token
  int more;          // the share goes on after it
  int last_share;    // the share that ends a block which this one begins and does not end
};
struct Walk {
  const PagedAttendParams& p;
  int Gq, TB;
  int64_t start, x1;  // first unit of the current block, end of the share
  __device__ __forceinline__ int blocks(const PagedReq& q) const { return (q.T + TB - 1) / TB; }
  __device__ __forceinline__ int tiles(const PagedReq& q, int blk) const {
    const int last = q.L - q.T + min(q.T, (blk + 1) * TB);  // rows the last token sees
    return max(1, (q.C + kN - 1) / kN + (max(last, 0) + kN - 1) / kN);
  }
  // Units of the request's first n blocks of one KV head. The tiles of full blocks are
  // n CT + sum_{b < n} floor((x + TB b) / 128) with x = L - T + TB + 127, a sum of floors
  // that needs no loop where TB divides 128 or is a multiple of it.
  __device__ __forceinline__ int64_t first_blocks(const PagedReq& q, int n) const {
    int64_t sum = 0;
    int b = 0;
    const int full = min(n, q.T / TB);
    const int x = q.L - q.T + TB + kN - 1, ct = (q.C + kN - 1) / kN;
    if (full > 2 && q.L >= q.T) {
      if (TB % kN == 0) {
        sum = (int64_t)full * (ct + x / kN) + (int64_t)(TB / kN) * full * (full - 1) / 2;
        b = full;
      } else if (kN % TB == 0) {
        // with x = 128 e + TB u + v, v < TB, block b has e + floor((u + b) / per), per = 128 / TB
        const int lg = __ffs(kN / TB) - 1, u = (x % kN) >> (7 - lg);  // per = 2^lg
        const int end = u + full, whole = end >> lg;  // sum of floor(i / per), u <= i < end
        sum = (int64_t)full * (ct + x / kN) + (((int64_t)whole * (whole - 1) / 2) << lg) +
              (int64_t)whole * (end - (whole << lg));
        b = full;
      }
    }
    for (; b < n; ++b) sum += tiles(q, b);
    return sum + (int64_t)n * kStart;
  }
  __device__ __forceinline__ int64_t request_units(const PagedReq& q) const {
    return first_blocks(q, blocks(q));
  }
  // The current block's tiles from unit `from` on, up to the share's end.
  __device__ __forceinline__ void set(Work& w, int64_t from) {
    w.n_tiles = tiles(w.q, w.blk);
    w.toks = min(TB, w.q.T - w.blk * TB);
    w.rows = w.toks * Gq;
    w.first = w.q.L - w.q.T + w.blk * TB;
    const int64_t tile0 = start + kStart, n = w.n_tiles;
    w.t0 = (int)min(max(from - tile0, (int64_t)0), n);
    w.t1 = (int)min(max(x1 - tile0, (int64_t)0), n);
    w.more = x1 > tile0 + n + kStart;  // the next block's first tile
  }
  __device__ __forceinline__ void enter(Work& w, int r) {
    int ignore = 0;
    w.r = r;
    w.q = paged_req(p, r, p.tc_rows, INT_MAX, &ignore);
    w.nb = blocks(w.q);
    w.CT = (w.q.C + kN - 1) / kN;
  }
  // The block that holds the share's first unit x0, `off` units into request r's. It may have no
  // tile left for the share.
  __device__ __forceinline__ void first_of(Work& w, int r, int64_t off, int64_t x0) {
    enter(w, r);
    const int64_t per_head = request_units(w.q);
    const bool small = ((off | per_head) >> 32) == 0;  // a 64-bit division is ten times a 32-bit one
    w.head = small ? (int)((uint32_t)off / (uint32_t)per_head) : (int)(off / per_head);
    const int64_t rem = off - w.head * per_head;
    int lo = 0, hi = w.nb;  // first_blocks(lo) <= rem < first_blocks(hi)
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_blocks(w.q, mid) <= rem) lo = mid;
      else hi = mid;
    }
    w.blk = lo;
    start = x0 - rem + first_blocks(w.q, lo);
    set(w, x0);
  }
  // The next block (whole warps; called only where w.more says that there is one).
  __device__ __forceinline__ void next(Work& w, int lane) {
    start += kStart + w.n_tiles;
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
    set(w, start);
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
  unsigned char* bounce = ring + NS * C::kTile;    // [8 warps][32 rows][128 bytes]
  uint64_t* bars = reinterpret_cast<uint64_t*>(bounce + 8 * kBounce);
  uint64_t* full = bars;            // [NS] ring tile landed
  uint64_t* empty = bars + NS;      // [NS] ring tile consumed
  // (each with one waiting party that sees every phase: entry 2 is half 0's, for the tiles of a
  // one-half block that use the second scores buffer)
  uint64_t* qfull = bars + 2 * NS;  // [2] a half's queries landed
  uint64_t* sfull = qfull + 2;      // [3] scores written
  uint64_t* pfull = qfull + 5;      // [3] probabilities written (128 threads)
  uint64_t* odone = qfull + 8;      // [2] a block's last P V of the half completed
  uint64_t* pdone = qfull + 10;     // a P V of a one-half block completed
  uint64_t* qempty = qfull + 11;    // [2] a block's last scores of the half formed
  uint64_t* bfull = qfull + 13;     // [kQueue] a block of the share announced
  uint64_t* bempty = bfull + kQueue;  // [kQueue] ... and done with (MMA warp, 8 softmax warps)
  uint64_t* phalf = bempty + kQueue;  // [3] the first half of the tile's probabilities written
  uint64_t* done = phalf + 3;         // every issued MMA completed
  __shared__ int64_t warp_tot[kThreads / 32];
  __shared__ int64_t start_off;
  __shared__ int start_r, cta_err;
  __shared__ int abort_word;
  __shared__ uint32_t tmem_holder;
  __shared__ Work blocks[kQueue];
  __shared__ int4 tail_item;
  __shared__ int tail_head;
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
      mbar_init(&qfull[h], 1);
      mbar_init(&qempty[h], 1);
      mbar_init(&odone[h], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], kHalf);
      mbar_init(&phalf[i], kHalf);
    }
    mbar_init(pdone, 1);
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&bfull[i], 1);
      mbar_init(&bempty[i], 9);
    }
    mbar_init(done, 1);
    abort_word = 0;
    cta_err = 0;
    tail_item = make_int4(-1, 0, 0, 0);
    tail_head = 0;
    start_r = -1;
    fence_mbar_init();
  }
  __syncthreads();

  // the CTA's share of the list: total tiles first, then the request that holds the share's start
  Walk walk{p, Gq, 2 * kHalf / Gq, 0, 0};
  int err = 0;
  int64_t total = 0, mine = 0;
  int G = 1;  // shares: no more than units, so that none inside a block is without a tile
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const int64_t x0 = pass ? total * blockIdx.x / G : 0;
    int64_t carry = 0;
    for (int r0 = 0; r0 < p.n_req; r0 += kThreads) {
      const int r = r0 + tid;
      int64_t v = mine;
      if (pass == 0 || p.n_req > kThreads) {
        v = 0;
        if (r < p.n_req)
          v = walk.request_units(paged_req(p, r, p.tc_rows, INT_MAX, &err)) * p.h_kv;
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
  walk.x1 = work ? total * (blockIdx.x + 1) / G : 0;

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
    uint32_t nb = 0;  // blocks of the share taken so far

    if (warp == 0) {
      // ---------------- walks the share, announces its blocks and copies their queries and tiles,
      // one page (or memory tile) and 64 dims a lane
      Work w;
      walk.first_of(w, start_r, start_off, x0);
      uint32_t seq = 0;
      const int ps = 1 << p.page_shift;
      const int br = min(ps, kN);               // rows of a box
      const int half = lane % SL, piece = lane / SL;
      struct Piece {  // what a lane copies of a tile
        bool load, ctx;
        int row;
        uint32_t bytes;  // of the whole tile
      };
      auto put = [&](const Piece& c, int kv) -> bool {  // the tile's K or V into the next slot
        const int s = seq % NS;
        if (seq >= NS) {
          bool free = true;
          if (lane == 0)
            free = wait_or_abort(&empty[s], ((seq / NS) - 1) & 1, &cta_err, abort_flag);
          if (!uniform(free)) return false;
        }
        ++seq;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], c.bytes);
        __syncwarp();
        if (c.load) {
          const CUtensorMap* m = c.ctx ? (kv ? &map_cv : &map_ck) : (kv ? &map_v : &map_k);
          tma3(ring + s * C::kTile + half * kSlice + piece * br * 128, m, half * 64, w.head, c.row,
               &full[s]);
        }
        return true;
      };
      bool ok = true;
      uint32_t n_blk[2] = {0, 0};  // blocks whose queries each half's barrier has seen
      bool was_two = false;
      // the rotated queries are written by the grid launched before this one
      asm volatile("griddepcontrol.wait;" ::: "memory");
      while (ok) {
        if (w.t0 == 0 && w.t1 < w.n_tiles) {  // goes on in the next shares: that of its last tile
          const int64_t end = walk.start + kStart + w.n_tiles;
          w.last_share = (int)((end * G + total - 1) / total - 1);
        }
        if (lane == 0) {
          const int b = nb % kQueue;
          ok = nb < kQueue || wait_or_abort(&bempty[b], (nb / kQueue - 1) & 1, &cta_err, abort_flag);
          if (ok) {
            blocks[b] = w;
            mbar_arrive(&bfull[b]);
          }
        }
        ++nb;
        ok = uniform(ok) != 0;
        if (!ok || w.t0 == w.t1) break;  // (a share without a tile: the others see as much)
        // the block's queries, once the scores of the block before are formed: a half's rows are
        // consecutive in each slice of its head's; one half's low parts take the other's place
        const bool two = w.rows > kHalf;
        if (lane == 0) {
          if (n_blk[0] > 0) ok = wait_or_abort(&qempty[0], (n_blk[0] - 1) & 1, &cta_err, abort_flag);
          if (was_two)
            ok = ok && wait_or_abort(&qempty[1], (n_blk[1] - 1) & 1, &cta_err, abort_flag);
        }
        ok = uniform(ok) != 0;
        if (!ok) break;
        was_two = two;
        ++n_blk[0];
        n_blk[1] += two;
        if (lane == 0) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int rows = two ? min(w.rows - h * kHalf, kHalf) : w.rows;
            uint64_t* bar = &qfull[two ? h : 0];
            if (two || h == 0)
              mbar_arrive_expect_tx(bar, (uint32_t)(rows * 128 * SL) * (two ? 1u : 2u));
            for (int sl = 0; sl < SL; ++sl)
              bulk_g2s(q_s + h * C::kTile + sl * kSlice,
                       p.q_rot + (((int64_t)((two ? 0 : h * p.h_kv) + w.head) * SL + sl) *
                                      p.n_rows * Gq +
                                  (int64_t)(w.q.a + w.blk * walk.TB) * Gq + (two ? h * kHalf : 0)) *
                                     64,
                       (uint32_t)rows * 128u, bar);
          }
        }
        __syncwarp();
        // K0 K1 V0 K2 V1 .. : a tile's V is needed a softmax after its K, and in a slot it takes up
        // from its copy's issue on
        Piece last{};
        for (int t = w.t0; ok && t < w.t1; ++t) {
          Piece cur;
          cur.ctx = t < w.CT;
          const int k0 = (cur.ctx ? t : t - w.CT) * kN;
          cur.row = 0;
          if (cur.ctx) {
            cur.load = piece == 0;
            cur.row = w.r * p.max_ctx + k0;
          } else {
            const int k = k0 + piece * br;
            cur.load = piece < kN / br && k < w.q.L;
            if (cur.load) {
              const int page = p.table[(int64_t)w.r * p.max_pages + (k >> p.page_shift)];
              if (page < 0 || page >= p.n_pages) {
                err = kErrBadIndex;
                cur.load = false;
              } else {
                cur.row = (page << p.page_shift) + (k & (ps - 1));
              }
            }
          }
          cur.bytes = __popc(__ballot_sync(0xffffffffu, cur.load)) *
                      (uint32_t)(cur.ctx ? kN : br) * 128u;
          ok = put(cur, 0) && (t == w.t0 || put(last, 1));
          last = cur;
        }
        ok = ok && put(last, 1);
        if (!w.more) break;
        walk.next(w, lane);
      }
      // the copies issued land before the CTA can exit
      for (int h = 0; h < 2; ++h)
        if (n_blk[h] > 0) mbar_wait_bounded(&qfull[h], (n_blk[h] - 1) & 1, &cta_err);
      for (uint32_t q = seq > NS ? seq - NS : 0; q < seq; ++q)
        mbar_wait_bounded(&full[q % NS], (q / NS) & 1, &cta_err);
    } else if (warp == 1) {
      // ---------------- MMA issuer: the warp stays converged, see mma_ss
      constexpr uint32_t idesc_s = (1u << 4) | (1u << 7) | (1u << 10) |
                                   ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(kHalf >> 4) << 24);
      constexpr uint32_t idesc_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                   ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kHalf >> 4) << 24);
      constexpr uint32_t kStep = C::kTile >> 4;  // ring tile in descriptor units
      const uint64_t q_desc = desc_k(q_s), k_desc = desc_k(ring), v_desc = desc_mn(ring);
      uint32_t seq = 0;              // ring tile of the block's first K
      uint32_t nq[2] = {0, 0}, np[3] = {0, 0, 0};
      auto wait = [&](uint64_t* bar, uint32_t par) {
        return uniform(wait_or_abort(bar, par, &cta_err, abort_flag)) != 0;
      };
      auto wait_ring = [&](uint32_t q) { return wait(&full[q % NS], (q / NS) & 1); };
      // (low: with the queries' low parts)
      auto scores = [&](int h, int slot, int bar, int st, bool low) {  // S[slot] = Q_h K^T
        fence_after();
        const uint64_t a = q_desc + h * kStep, b = k_desc + st * kStep;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {  // 16 dims a step: 32 bytes of a row, 64 dims a slice
          const uint32_t off = (kk >> 2) * (kSlice >> 4) + 2 * (kk & 3);
          mma_ss(tmem + slot * 128, a + off, b + off, idesc_s, kk ? 1u : 0u);
        }
        if (low) {
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            const uint32_t off = (kk >> 2) * (kSlice >> 4) + 2 * (kk & 3);
            mma_ss(tmem + slot * 128, a + kStep + off, b + off, idesc_s, 1u);
          }
        }
        commit(&sfull[bar]);
      };
      // O_h (+)= P[slot] V as the two halves of the tile's probabilities are written
      auto product = [&](int h, int slot, int bar, uint32_t par, int st, bool first) {
        const uint64_t b = v_desc + st * kStep;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!wait(hf ? &pfull[bar] : &phalf[bar], par)) return false;
          fence_after();
#pragma unroll
          for (int kk = hf * 4; kk < hf * 4 + 4; ++kk)  // 16 keys a step
            mma_ts(tmem + 256 + h * 128, tmem + slot * 128 + kk * 8, b + kk * (2048 >> 4), idesc_o,
                   (first && kk == 0) ? 0u : 1u);
        }
        return true;
      };
      bool ok = true;
      while (true) {
        const int bq = nb % kQueue;
        if (!wait(&bfull[bq], (nb / kQueue) & 1)) break;
        ++nb;
        const int n = uniform(blocks[bq].t1 - blocks[bq].t0);
        const bool two = uniform(blocks[bq].rows) > kHalf, more = uniform(blocks[bq].more) != 0;
        if (lane == 0) mbar_arrive(&bempty[bq]);
        if (n == 0) break;
        if (two) {
          // two halves in alternation, each with its own scores
          ok = wait_ring(seq);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && wait(&qfull[h], nq[h] & 1);
            ++nq[h];
            if (ok) scores(h, h, h, seq % NS, false);
            if (ok && n == 1) commit(&qempty[h]);
          }
          if (!ok) break;
          commit(&empty[seq % NS]);
#pragma unroll 1
          for (int j = 0; j < n; ++j) {
            const bool last = j + 1 == n;
            const uint32_t k = seq + 2 * j + 1, v = last ? k : k + 1;  // next K, this V
            // both first: what follows the probabilities is the critical path
            ok = wait_ring(v) && (last || wait_ring(k)) &&
                 product(0, 0, 0, np[0] & 1, v % NS, j == 0);
            ++np[0];
            if (!ok) break;
            if (last) {
              commit(&odone[0]);
            } else {
              scores(0, 0, 0, k % NS, false);
              if (j + 2 == n) commit(&qempty[0]);
            }
            ok = product(1, 1, 1, np[1] & 1, v % NS, j == 0);
            ++np[1];
            if (!ok) break;
            commit(&empty[v % NS]);
            if (last) {
              commit(&odone[1]);
            } else {
              scores(1, 1, 1, k % NS, false);
              if (j + 2 == n) commit(&qempty[1]);
              commit(&empty[k % NS]);
            }
          }
        } else {
          // one half: its scores alternate between both buffers, a tile ahead of the products
          ok = wait_ring(seq) && wait(&qfull[0], nq[0] & 1);
          ++nq[0];
          if (!ok) break;
          scores(0, 0, 0, seq % NS, true);
          if (n == 1) commit(&qempty[0]);
          commit(&empty[seq % NS]);
#pragma unroll 1
          for (int j = 0; j < n; ++j) {
            const int slot = j & 1;
            const bool last = j + 1 == n;
            const uint32_t k = seq + 2 * j + 1, v = last ? k : k + 1;
            if (!last) {
              ok = wait_ring(k);
              if (!ok) break;
              scores(0, slot ^ 1, slot ? 0 : 2, k % NS, true);
              if (j + 2 == n) commit(&qempty[0]);
              commit(&empty[k % NS]);
            }
            ok = wait_ring(v) &&
                 product(0, slot, 2 * slot, (slot ? np[2] : np[0]) & 1, v % NS, j == 0);
            if (slot) ++np[2];
            else ++np[0];
            if (!ok) break;
            commit(&empty[v % NS]);
            commit(pdone);
            if (last) commit(&odone[0]);
          }
        }
        seq += 2 * n;
        if (!ok || !more) break;
      }
      commit(done);
      mbar_wait_bounded(done, 0, &cta_err);
    } else {
      // ---------------- softmax: a half's 128 rows, one a thread
      const int h = (warp - 2) >> 2;
      const int lrow = (warp & 3) * 32 + lane;        // row in the half = TMEM lane
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t o_col = lane_base + 256 + h * 128;
      const float c = p.scale_log2;
      const int row = h * kHalf + lrow, row_tok = row / Gq;  // row of a block, its token
      uint32_t n_own = 0, n_alt = 0;  // phases of sfull[h], of sfull[2]
      uint32_t no = 0, npd = 0;       // of odone[h], of pdone
      uint32_t seq = 0;            // ring tile of the block's first K
      auto wait = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, par, &cta_err, abort_flag));
      };
      bool ok = true;
      while (true) {
        // the block's geometry stays in shared memory: the tile loop holds a row of scores in
        // registers
        ok = wait(&bfull[nb % kQueue], (nb / kQueue) & 1);
        if (!ok) break;
        const Work& w = blocks[nb % kQueue];
        const bool two = w.rows > kHalf;
        const bool active = h == 0 || two;
        if (w.t0 == w.t1) break;
        const int t0 = w.t0, t1 = w.t1, CT = w.CT, n_ctx = w.q.C, n_loc = w.q.L;
        const bool more = w.more != 0;
        const bool any_row = h * kHalf + (warp & 3) * 32 < w.rows;  // of the warp
        float m = -INFINITY, l = 0.f;
        if (active) {
          // last visible local row of this row and of the half's first
          const int vis = w.first + min(row_tok, w.toks - 1);
          const int vis_first = min(w.first + h * (walk.TB >> 1), n_loc - 1);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          for (int t = t0; t < t1; ++t) {
            const bool ctx = t < CT;
            const int k0 = (ctx ? t : t - CT) * kN;
            const int valid = (ctx ? n_ctx : n_loc) - k0;            // rows the tile holds
            const bool alt = !two && ((t - t0) & 1);   // the second scores buffer
            const int bar = alt ? 2 : h;
            const uint32_t s_col = lane_base + (alt ? 128 : h * 128);
            const uint32_t par = (alt ? n_alt++ : n_own++) & 1;
            ok = p.wait_limit == 0
                     ? wait(&sfull[bar], par)
                     : __all_sync(0xffffffffu, poll_or_abort(&sfull[bar], par, p.wait_limit,
                                                             &cta_err, abort_flag));
            if (!ok) break;
            fence_after();
            // V rows past the end hold anything: cleared, for 0 * NaN would reach O
            if (h == 0 && valid < kN) {
              const uint32_t q = seq + 2 * (t - t0) + (t + 1 == t1 ? 1 : 2);
              ok = wait(&full[q % NS], (q / NS) & 1);
              if (!ok) break;
              unsigned char* v = ring + (q % NS) * C::kTile;
              const int at = max(valid, 0) * 128;   // every thread of the half 16 bytes a step
#pragma unroll 1
              for (int i = at + lrow * 16; i < (int)kSlice; i += kHalf * 16)
#pragma unroll
                for (int sl = 0; sl < SL; ++sl)
                  *reinterpret_cast<uint4*>(v + sl * kSlice + i) = make_uint4(0u, 0u, 0u, 0u);
              fence_proxy_async_smem();
            }
            if (any_row) {
              float sr[128];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                ld32(s_col + i * 32, reinterpret_cast<uint32_t*>(sr) + i * 32);
              wait_ld();
              if (!(ctx ? valid >= kN : k0 + kN - 1 <= vis_first)) {
                const int lim = min(valid - 1, ctx ? kN : vis - k0);  // keys [0, lim] visible
#pragma unroll
                for (int i = 0; i < 128; ++i)
                  if (i > lim) sr[i] = -INFINITY;
              }
              float mx[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = max3(sr[e], sr[e + 4], sr[e + 8]);
#pragma unroll
              for (int i = 12; i < 124; i += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], sr[i + e], sr[i + 4 + e]);
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], sr[124 + e]);
              const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
              const bool raise = mt > m + kRaise || (m == -INFINITY && mt != -INFINITY);
              if (__any_sync(0xffffffffu, raise)) {
                const float mn = raise ? mt : m;
                const float alpha = (raise && m != -INFINITY) ? ex2(m - mn) : 1.f;
                m = mn;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  sum[e].x *= alpha;
                  sum[e].y *= alpha;
                }
                if (t > t0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                  if (!two) {  // the previous product may still run (two halves: it cannot)
                    ok = wait(pdone, (npd + (t - t0) - 1) & 1);
                    if (!ok) break;
                    fence_after();
                  }
#pragma unroll 1
                  for (int ch = 0; ch < D / 16; ++ch) {
                    uint32_t ov[16];
                    ld16(o_col + ch * 16, ov);
                    wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                      ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                    st16(o_col + ch * 16, ov);
                  }
                }
              }
              // the probabilities in bf16 over the scores' columns (their sum in fp32)
              const float neg = m == -INFINITY ? 0.f : -m;
              const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
#pragma unroll
              for (int ch = 0; ch < 8; ++ch) {
                uint32_t pk[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  float2 x = __ffma2_rn(make_float2(sr[ch * 16 + 2 * i], sr[ch * 16 + 2 * i + 1]),
                                        c2, n2);
                  x.x = ex2(x.x);
                  x.y = ex2(x.y);
                  sum[i & 1] = __fadd2_rn(sum[i & 1], x);
                  pk[i] = pack_bf16(x.x, x.y);
                }
                st8(s_col + ch * 8, pk);
                if (ch == 3) {
                  wait_st();
                  fence_before();
                  mbar_arrive(&phalf[bar]);
                }
              }
              wait_st();
            } else {
              mbar_arrive(&phalf[bar]);
            }
            fence_before();
            mbar_arrive(&pfull[bar]);
          }
          l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        const int n = t1 - t0;
        seq += 2 * n;
        if (!two) npd += n;
        if (!ok) break;
        const bool begins = t0 == 0, ends = t1 == w.n_tiles;
        if (active) {
          ok = wait(&odone[h], no++ & 1);
          if (!ok) break;
          fence_after();
          const bool whole = begins && ends;
          // A lane holds a row: its 128-byte pieces go through shared memory (16-byte chunk c of
          // row r at c ^ (r & 7)), so that eight lanes write a piece of one row together.
          if (any_row) {
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const int64_t pslot = ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * (2 * kHalf);
            unsigned char* dst =
                whole ? reinterpret_cast<unsigned char*>(
                            static_cast<__nv_bfloat16*>(p.O) +
                            ((int64_t)(w.q.a + w.blk * walk.TB) * p.h_q + w.head * Gq) * D)
                      : reinterpret_cast<unsigned char*>(p.tc_o + pslot * D);
            dst += (lane & 7) * 16;
            // the row's place: query head row - row_tok Gq of its group, or a row of the partial
            const uint32_t off = whole ? (uint32_t)((row_tok * (p.h_q - Gq) + row) * D * 2)
                                       : (uint32_t)(row * D * 4);
            unsigned char* mine = bounce + (warp - 2) * kBounce;
            const int n_row = w.rows - (row - lane);             // the warp's rows
            const int steps = whole ? D / 64 : D / 32;
#pragma unroll 1
            for (int st = 0; st < steps; ++st, dst += 128) {
              uint32_t ov[32];
              if (whole) {
                uint32_t f[64];
                ld32(o_col + st * 64, f);
                ld32(o_col + st * 64 + 32, f + 32);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  ov[i] = pack_bf16(__uint_as_float(f[2 * i]) * inv,
                                    __uint_as_float(f[2 * i + 1]) * inv);
              } else {
                ld32(o_col + st * 32, ov);
                wait_ld();
              }
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(mine + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                    make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
              __syncwarp();
              uint4 v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3);
                v[i] = *reinterpret_cast<const uint4*>(mine + r * 128 +
                                                       (((lane & 7) ^ (r & 7)) << 4));
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3);
                const uint32_t to = __shfl_sync(0xffffffffu, off, r);
                if (r < n_row) *reinterpret_cast<uint4*>(dst + to) = v[i];
              }
              __syncwarp();
            }
            if (!whole && lane < n_row)
              *reinterpret_cast<float2*>(p.tc_ml + (pslot + row) * 2) = make_float2(m, l);
          }
          fence_before();  // O is read before the next block's products
        }
        if (begins && !ends && tid == 64) {  // goes on in the next CTAs' shares
          tail_item = make_int4(w.q.a, w.q.T, w.blk, w.last_share);
          tail_head = w.head;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bempty[nb % kQueue]);  // the block has been read
        ++nb;
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
  if (tid == 0) {
    if (cta_err == kErrWaitTimeout) tail_item.x = -1;
    p.tc_tail[2 * blockIdx.x] = tail_item;
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
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = allow_smem_once(reinterpret_cast<const void*>(kfn), Cfg<D>::smem, ready);
  if (e != cudaSuccess) return e;
  return launch_early(kfn, dim3(grid), dim3(kThreads), Cfg<D>::smem, st, mk, mv, mck, mcv, p);
}

}  // namespace pgt

cudaError_t launch_paged_attend_tc(const PagedAttendParams& p, int grid, int d, cudaStream_t st) {
  return d == 128 ? pgt::launch<128>(p, grid, st) : pgt::launch<64>(p, grid, st);
}

}  // namespace msa
