// paged_attend.cu - attention of ragged requests over [routed memory ; paged local context]: the
// operation of sparse generation
//   [news.neo-ai.one article, "グローバル RoPE（アクティブコンテキスト）" and "推論パイプライン";
//    ruixiangma.github.io blog, "三阶段推理流程"]
// for a batch whose requests differ in length, with their local K/V in pages of one pool. Token i
// of request r's T new ones sits at local row j = len - T + i; its query, rotated at pos0 + j,
// attends over the request's memory rows and its local rows <= j (keys stored rotated):
//   O = softmax(scale q . k) v, 0 where nothing is visible.
//
// The kernel of this file streams each key row once per 16 query rows (bf16: 8) and is the one for
// few query rows per KV head (single tokens) and for fp32. A warp works alone: for one KV head it
// takes a contiguous range of the flattened list (request, block of query rows, tile of keys),
// copies the tiles with cp.async into its own ring in shared memory (no barrier between warps), forms the scores and P V with warp-level MMAs (bf16; fp32 as three tf32 products of
// the operands' high and low parts) and keeps the running maximum and sum of the softmax in
// registers. All ranges of a head have the same number of tiles to within one, whatever the
// requests' lengths; consecutive warps take the KV heads of the same range, so their copies
// cover whole key rows. A query block that a range does not hold whole leaves a partial
// (m, l, o), which the merge kernel folds in the order of the ranges (no atomics: a call's
// result does not depend on timing). Bound by HBM for single tokens.
#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"
#include "paged.cuh"

namespace msa {
namespace pga {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
template <typename T> constexpr int kBlockRows = sizeof(T) == 2 ? kPagedWarpRows : 16;
constexpr int kRing = 24576;        // bytes of a warp's ring
constexpr int kMinTiles = 2;        // a range is at least this many tiles
constexpr int kAngles = 2048;       // bytes of a warp's angle table: the tokens of a query block
constexpr int kReqCache = 256;      // requests whose geometry is kept in shared memory
constexpr int kMergeThreads = 256;
constexpr size_t kMaxSmem =
    kWarps * (size_t)(kRing + kAngles) + (kPagedMaxReq + 1) * sizeof(int32_t);

template <typename T, int D> struct Geo {
  // keys of a tile: 8 KB of K and V (16 keys at bf16, d = 64, paid the softmax's shuffles and the
  // copies' bookkeeping for 4 KB)
  static constexpr int KT = sizeof(T) == 2 ? 2048 / D : 8;
  static constexpr int MIN_TILES = sizeof(T) == 2 ? kMinTiles : 3 * kMinTiles;
  static constexpr int RB = D * (int)sizeof(T);            // bytes of a key row of one head
  static constexpr int TILE = KT * RB;                     // K (or V) of a tile
  static constexpr int NST = kRing / (2 * TILE);           // stages of the ring
};

__device__ __forceinline__ float ex2(float x) {  // max relative error 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp16_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float lds32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// a pair of values as bf16 high parts and what they leave, rounded to bf16: 2^-17 of the value
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x, y);
  lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
}
// x = hi + lo with both in tf32 (11 significant bits each): hi hi + hi lo + lo hi leaves out
// lo lo, 2^-22 of the product, next to fp32's own 2^-24
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  const float rest = x - __uint_as_float(hi);
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
}

// A sum of products with the operands' high parts plus those with the low parts. An infinite
// operand has an infinite high part, whose products are what they should be, and a low part of
// NaN, and the other operand's low part may have any sign or be 0: the low sum is left out where
// it makes NaN of the high one.
__device__ __forceinline__ float add_low(float hi, float lo) {
  const float s = hi + lo;
  return s == s ? s : hi;
}

template <int KT> __device__ __forceinline__ int ctx_tiles(const PagedReq& q) {
  return (q.C + KT - 1) / KT;
}
// tiles of a query block (at least one, so that a block that sees nothing is still written)
template <int KT> __device__ __forceinline__ int block_tiles(const PagedReq& q) {
  return max(1, ctx_tiles<KT>(q) + (int)(((long long)q.L + KT - 1) / KT));
}

// range s of S over x tiles: [s x / S, (s + 1) x / S); range_of(y) is the range that holds tile y
__device__ __forceinline__ int64_t range_start(int64_t x, int s, int S) { return x * s / S; }
__device__ __forceinline__ int range_of(int64_t y, int64_t x, int S) {
  return (int)(((y + 1) * S + x - 1) / x - 1);
}

// The queries of the requests that the tcgen05 kernel serves, rotated and rounded to bf16, in
// its operand layout: per KV head and 64 dims the rows (token, query head of the group) one after
// another, 16-byte chunk c of a row at c ^ (row within its block & 7). A warp takes 16 heads of a
// token (their loads in flight together): its angles once into the warp's table, then a lane one
// 16-byte chunk of the lower half of a head and its partner half a head on. What rounding to bf16
// leaves follows in a second copy, for the blocks that take it.
template <int D>
__device__ __forceinline__ void rotate_queries(const PagedAttendParams& p, int w, int n_warps,
                                               int lane, float2* table,
                                               const unsigned long long* turns) {
  constexpr int HC = D / 16;       // chunks of half a head
  constexpr int HPW = 32 / HC;     // heads a warp takes at once
  constexpr int NI = 16 / HPW;
  const int Gq = p.h_q / p.h_kv, TB = 256 / Gq;
  const int c = lane % HC;
  const int64_t rows = (int64_t)p.n_rows * Gq;
  const int parts = (p.h_q + 15) / 16;
#pragma unroll 1
  for (int64_t unit = w; unit < (int64_t)p.n_rows * parts; unit += n_warps) {
    const int i = (int)(unit / parts), h0 = (int)(unit % parts) * 16 + lane / HC;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.Q) + i * p.q_stride + c * 8;
    uint4 ra[NI], rb[NI];
#pragma unroll
    for (int k = 0; k < NI; ++k) {  // (any row of Q may be read, whoever it belongs to)
      const int h = min(h0 + k * HPW, p.h_q - 1);
      ra[k] = *reinterpret_cast<const uint4*>(src + h * D);
      rb[k] = *reinterpret_cast<const uint4*>(src + h * D + D / 2);
    }
    int lo = 0, hi = p.n_req;      // the request of token i: row_start[lo] <= i < row_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.row_start[mid] <= i) lo = mid;
      else hi = mid;
    }
    int ignore = 0;
    const PagedReq q = paged_req(p, lo, p.tc_rows, INT_MAX, &ignore);
    const int t = i - q.a;
    if (t < 0 || t >= q.T) continue;
    const int64_t pos = (int64_t)p.pos0 + q.L - q.T + t;
#pragma unroll 1
    for (int e = lane; e < D / 2; e += 32)
      table[e] = p.rope ? rot_turns(pos, turns[e]) : make_float2(1.f, 0.f);
    __syncwarp();
    float4 cs[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = *reinterpret_cast<const float4*>(table + c * 8 + 2 * e);
    const int x0 = (t % TB) * Gq;
    const bool low = min(TB, q.T - t / TB * TB) * Gq <= 128;  // a block of one half
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      const int h = h0 + k * HPW;
      if (h >= p.h_q) break;
      using V = Vec<__nv_bfloat16, 8>;
      float a[8], b[8];
      V::unpack(ra[k], a);
      V::unpack(rb[k], b);
      uint32_t oa[4], ob[4], la[4], lb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        split_bf16(a[2 * e] * cs[e].x - b[2 * e] * cs[e].y,
                   a[2 * e + 1] * cs[e].z - b[2 * e + 1] * cs[e].w, oa[e], la[e]);
        split_bf16(b[2 * e] * cs[e].x + a[2 * e] * cs[e].y,
                   b[2 * e + 1] * cs[e].z + a[2 * e + 1] * cs[e].w, ob[e], lb[e]);
      }
      const int kv = h / Gq, g = h % Gq;
      const int x = (x0 + g) & 7;
      __nv_bfloat16* dst =
          p.q_rot + ((int64_t)kv * (D / 64) * rows + (int64_t)i * Gq + g) * 64;
      const int cb = c + HC;  // D = 64: the same 64 dims; D = 128: the next ones
      const int64_t oa_at = (c ^ x) << 3, ob_at = (cb >> 3) * rows * 64 + (((cb & 7) ^ x) << 3);
      *reinterpret_cast<uint4*>(dst + oa_at) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
      *reinterpret_cast<uint4*>(dst + ob_at) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
      if (low) {
        dst += (int64_t)p.h_q * p.n_rows * D;
        *reinterpret_cast<uint4*>(dst + oa_at) = make_uint4(la[0], la[1], la[2], la[3]);
        *reinterpret_cast<uint4*>(dst + ob_at) = make_uint4(lb[0], lb[1], lb[2], lb[3]);
      }
    }
    __syncwarp();  // the table is filled anew
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) paged_attend_kernel(PagedAttendParams p, int S_max) {
  using G = Geo<T, D>;
  constexpr int KT = G::KT, RB = G::RB, TILE = G::TILE, NST = G::NST;
  constexpr bool BF = sizeof(T) == 2;
  // query rows of a block: the MMA's 16, or (bf16) 8 with their high parts as the MMA's rows 0-7
  // and their low parts as its rows 8-15, so that neither the rotated queries nor the
  // probabilities lose to bf16 what a single part would (the tensor cores' work is the same, and
  // decode has few rows)
  constexpr int kRows = kBlockRows<T>;
  constexpr int HR = kRows / 8;                  // rows of a lane
  constexpr int NT = D / 8;                      // 8-wide output tiles
  constexpr int KS = BF ? D / 16 : D / 8;        // k steps of the scores
  extern __shared__ __align__(128) unsigned char sm_raw[];
  int32_t* pre = reinterpret_cast<int32_t*>(sm_raw + kWarps * (kRing + kAngles));  // [n_req + 1]
  // requests as paged_req has them, where they are few (the space a longer prefix list takes)
  PagedReq* reqs = reinterpret_cast<PagedReq*>(pre + kReqCache + 4);
  __shared__ int64_t warp_tot[kWarps];
  __shared__ int cta_err;
  // the angles' fractions, read lane by lane (from the parameters that is a load per lane)
  __shared__ unsigned long long turns[D / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Gq = p.h_q / p.h_kv;
  if (tid < D / 2) turns[tid] = p.rope_turns[tid];

  wait_then_let_start();  // the tcgen05 kernel or the merge, which wait for the results
  if (tid == 0) cta_err = 0;
  __syncthreads();
  int err = 0;
  // first tile of every request in the flattened list of one KV head
  int64_t carry = 0;
  for (int r0 = 0; r0 < p.n_req; r0 += kThreads) {
    const int r = r0 + tid;
    int64_t v = 0;
    if (r < p.n_req) {
      const PagedReq q = paged_req(p, r, 0, p.tc_rows, &err);
      if (p.n_req <= kReqCache) reqs[r] = q;
      v = (int64_t)(((long long)q.T * Gq + kRows - 1) / kRows) * block_tiles<KT>(q);
    }
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int64_t base = carry;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += warp_tot[w];
      carry += warp_tot[w];
    }
    if (r < p.n_req) pre[r] = (int32_t)(base + inc - v);
    __syncthreads();
  }
  if (tid == 0) pre[p.n_req] = (int32_t)carry;
  __syncthreads();
  // (A list of 2^31 tiles is refused: its prefix sums are 32-bit, for as many of 64 bits do not
  // fit beside the rings.)
  if (carry > INT_MAX) err = kErrCtxOverflow;
  const int64_t total = carry > INT_MAX ? 0 : carry;
  const int S = (int)max((int64_t)1, min((int64_t)S_max, total / G::MIN_TILES));
  const int w_all = blockIdx.x * kWarps + warp;
  const int s = w_all / p.h_kv, head = w_all % p.h_kv;
  const int64_t x0 = s < S ? range_start(total, s, S) : total;
  const int64_t x1 = s < S ? range_start(total, s + 1, S) : total;
  const int n_tiles = (int)(x1 - x0);
  int4 tail = make_int4(-1, 0, 0, 0);

  if (n_tiles > 0) {
    const uint32_t ring = smem_u32(sm_raw) + warp * kRing;
    // where a tile of the list lies
    struct Cur {
      int r, blk, t, TPP, CT, nb;
      int last;  // last local row that the block's last token sees
      PagedReq q;
    };
    auto set_last = [&](Cur& c) {
      c.last = min(c.q.L - c.q.T + min((c.blk * kRows + kRows - 1) / Gq, c.q.T - 1), c.q.L - 1);
    };
    auto enter = [&](Cur& c, int r) {  // request r's geometry (r has tiles)
      int ignore = 0;
      c.r = r;
      c.q = p.n_req <= kReqCache ? reqs[r] : paged_req(p, r, 0, p.tc_rows, &ignore);
      c.CT = ctx_tiles<KT>(c.q);
      c.TPP = block_tiles<KT>(c.q);
      c.nb = (int)(((long long)c.q.T * Gq + kRows - 1) / kRows);
    };
    auto step = [&](Cur& c) {  // the next tile of the list (only called when there is one)
      if (++c.t < c.TPP) return;
      c.t = 0;
      if (++c.blk == c.nb) {
        c.blk = 0;
        int r = c.r + 1;
        while (pre[r + 1] == pre[r]) ++r;
        enter(c, r);
      }
      set_last(c);
    };
    Cur ld;
    {
      int lo = 0, hi = p.n_req;  // last request whose first tile is <= x0
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x0) lo = mid;
        else hi = mid;
      }
      enter(ld, lo);
      const int off = (int)x0 - pre[lo];
      ld.blk = off / ld.TPP;
      ld.t = off % ld.TPP;
      set_last(ld);
    }
    Cur cu = ld;  // the tile being computed; ld is the tile being loaded

    // The block table of the request being loaded, 32 entries at a time: lane i holds that of
    // page win + i.
    int win = 0, window = 0;
    auto look = [&](const Cur& c, bool entered) {  // the window holds the pages of c's tile
      if (c.t < c.CT) return;
      const int pg = ((c.t - c.CT) * KT) >> p.page_shift;
      if (!entered && pg - win >= 0 && pg - win < 31) return;
      win = pg;
      window = p.table[(int64_t)c.r * p.max_pages + min(pg + lane, p.max_pages - 1)];
    };
    look(ld, true);
    int looked = ld.r;  // request the window belongs to (-1: none yet)
    if (ld.t < ld.CT) looked = -1;
    auto issue = [&](int v) {  // copies of tile v of the range into stage v % NST
      const Cur& c = ld;
      const uint32_t st = ring + (uint32_t)(v % NST) * (2 * TILE);
      const int64_t pitch = (int64_t)p.h_kv * RB;
      // byte offsets of the tile's first row, and of its 17th less 16 rows, in the source
      int64_t at[2] = {0, 0};
      const char* ks = nullptr;
      const char* vs = nullptr;
      int valid = 0;
      if (c.t < c.CT) {
        at[0] = at[1] = (((int64_t)c.r * p.max_ctx + c.t * KT) * p.h_kv + head) * RB;
        ks = static_cast<const char*>(p.cK);
        vs = static_cast<const char*>(p.cV);
        valid = min(KT, c.q.C - c.t * KT);
      } else {
        const int k0 = (c.t - c.CT) * KT;
        if (k0 <= c.last) {
          look(c, looked != c.r);
          looked = c.r;
          valid = min(KT, c.q.L - k0);
          bool ok = true;
#pragma unroll
          for (int e = 0; e < (KT > 16 ? 2 : 1); ++e) {
            const int k = k0 + 16 * e;  // pages hold 16 rows or more
            const int page = __shfl_sync(0xffffffffu, window, (k >> p.page_shift) - win);
            if (16 * e < valid && (page < 0 || page >= p.n_pages)) ok = false;
            at[e] = ((((int64_t)page << p.page_shift) + (k & ((1 << p.page_shift) - 1)) - 16 * e) *
                         p.h_kv +
                     head) * RB;
          }
          if (ok) {
            ks = static_cast<const char*>(p.K_pages);
            vs = static_cast<const char*>(p.V_pages);
          } else {
            err = kErrBadIndex;
          }
        }
      }
      if (ks != nullptr) {  // rows past the end are filled with zeros (their V meets P = 0)
        constexpr int CPR = RB / 16;      // 16-byte chunks of a row
        constexpr int RPI = 32 / CPR;     // rows a warp instruction copies
        const int c16 = lane % CPR, r0 = lane / CPR;
#pragma unroll
        for (int i = 0; i < KT / RPI; ++i) {
          const int row = r0 + i * RPI;
          const bool ok = row < valid;
          const int64_t off = ok ? at[i * RPI >= 16 ? 1 : 0] + row * pitch + c16 * 16 : 0;
          const uint32_t dst = st + row * RB + ((c16 ^ (row & 7)) << 4);
          cp16_zfill(dst, ks + off, ok);
          cp16_zfill(dst + TILE, vs + off, ok);
        }
      }
      if (v + 1 < n_tiles) step(ld);
    };
#pragma unroll
    for (int v = 0; v < NST - 1; ++v) {
      if (v < n_tiles) issue(v);
      cp_commit();
    }

    const int gr = lane >> 2, t4 = lane & 3;
    uint32_t qh[KS][4];                       // query fragments (bf16, or tf32 high parts)
    uint32_t ql[BF ? 1 : KS][4];              // fp32: low parts
    float o[NT][4];
    float m[HR], l[HR];
    int v = 0;
    while (v < n_tiles) {
      // ---- one query block's share of the range
      const bool begins = cu.t == 0;
      const int t_end = (int)min((int64_t)cu.TPP, (int64_t)cu.t + (n_tiles - v));
      const bool ends = t_end == cu.TPP;
      const int nrow = min(kRows, (int)min((long long)kRows, (long long)cu.q.T * Gq - (long long)cu.blk * kRows));
      // The block's queries, rotated. A lane's fragment elements of dims i and i + D/2 are its
      // own, and the angles of a token are the same for all its heads: the warp computes them
      // once into a table in shared memory, CAP tokens at a time (the first exactly, the next
      // ones by rotating on: at most 3 steps of 2^-23 at d = 128, 7 at d = 64).
      int vis[HR], row_tok[HR];  // last local row that query rows gr (+ 8) see; their tokens
      const int tok0 = cu.blk * kRows / Gq;
      const int n_tok = (cu.blk * kRows + nrow - 1) / Gq - tok0 + 1;
#pragma unroll
      for (int hf = 0; hf < HR; ++hf) {
        const int row = cu.blk * kRows + min(gr + 8 * hf, nrow - 1);
        const int tok = row / Gq;
        vis[hf] = cu.q.L - cu.q.T + tok;
        row_tok[hf] = tok - tok0;
        const T* src = static_cast<const T*>(p.Q) + (int64_t)(cu.q.a + tok) * p.q_stride +
                       (head * Gq + row % Gq) * D;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)  // the values as stored; turned below
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qh[kk][hf + 2 * e] = *reinterpret_cast<const uint32_t*>(
                BF ? src + kk * 16 + e * 8 + 2 * t4 : src + kk * 8 + e * 4 + t4);
            if constexpr (BF) qh[kk][1 + 2 * e] = 0u;  // low parts
          }
      }
      if (p.rope) {
        constexpr int PL = D / 64;                  // RoPE pairs of a lane: l, l + 32
        constexpr int CAP = kAngles / (D / 2 * 8);  // tokens the table holds
        float2* table = reinterpret_cast<float2*>(sm_raw + kWarps * kRing + warp * kAngles);
        float2 cs[PL], st[PL];
#pragma unroll 1
        for (int t0 = 0; t0 < n_tok; t0 += CAP) {
          const int64_t pos = (int64_t)p.pos0 + cu.q.L - cu.q.T + tok0 + t0;
#pragma unroll
          for (int e = 0; e < PL; ++e) {
            cs[e] = rot_turns(pos, turns[lane + 32 * e]);
            if (n_tok > 1) st[e] = rot_turns(1, turns[lane + 32 * e]);
          }
#pragma unroll 1
          for (int t = 0; t < min(CAP, n_tok - t0); ++t) {
#pragma unroll
            for (int e = 0; e < PL; ++e) {
              table[t * (D / 2) + lane + 32 * e] = cs[e];
              if (n_tok > 1)
                cs[e] = make_float2(cs[e].x * st[e].x - cs[e].y * st[e].y,
                                    cs[e].y * st[e].x + cs[e].x * st[e].y);
            }
          }
          __syncwarp();
#pragma unroll
          for (int hf = 0; hf < HR; ++hf) {
            const int t = row_tok[hf] - t0;
            if (t < 0 || t >= CAP) continue;
            const float2* ang = table + t * (D / 2);
#pragma unroll
            for (int kk = 0; kk < KS / 2; ++kk) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t& lo = qh[kk][hf + 2 * e];           // dims i
                uint32_t& hi = qh[kk + KS / 2][hf + 2 * e];  // and i + D / 2
                if constexpr (BF) {
                  const float4 c = *reinterpret_cast<const float4*>(ang + kk * 16 + e * 8 + 2 * t4);
                  const float a0 = __uint_as_float(lo << 16), a1 = __uint_as_float(lo & 0xFFFF0000u);
                  const float b0 = __uint_as_float(hi << 16), b1 = __uint_as_float(hi & 0xFFFF0000u);
                  split_bf16(a0 * c.x - b0 * c.y, a1 * c.z - b1 * c.w, lo, qh[kk][1 + 2 * e]);
                  split_bf16(b0 * c.x + a0 * c.y, b1 * c.z + a1 * c.w, hi,
                             qh[kk + KS / 2][1 + 2 * e]);
                } else {
                  const float2 c = ang[kk * 8 + e * 4 + t4];
                  const float a = __uint_as_float(lo), b = __uint_as_float(hi);
                  lo = __float_as_uint(a * c.x - b * c.y);
                  hi = __float_as_uint(b * c.x + a * c.y);
                }
              }
            }
          }
          __syncwarp();  // the table is filled anew
        }
      }
      if constexpr (!BF) {
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = __uint_as_float(qh[kk][e]);
            split_tf32(x, qh[kk][e], ql[kk][e]);
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
#pragma unroll
      for (int hf = 0; hf < HR; ++hf) {
        m[hf] = -INFINITY;
        l[hf] = 0.f;
      }
      const int first_vis = cu.q.L - cu.q.T + cu.blk * kRows / Gq;  // of the block's first token

      for (; cu.t < t_end; ++cu.t, ++v) {
        cp_wait<NST - 2>();
        __syncwarp();
        if (v + NST - 1 < n_tiles) issue(v + NST - 1);
        cp_commit();
        const bool ctx = cu.t < cu.CT;
        const int k0 = ctx ? cu.t * KT : (cu.t - cu.CT) * KT;
        if (!ctx && k0 > cu.last) continue;  // nothing visible
        const bool full = ctx ? k0 + KT <= cu.q.C : k0 + KT - 1 <= first_vis;
        const uint32_t kb = ring + (uint32_t)(v % NST) * (2 * TILE), vb = kb + TILE;
        constexpr int NK = KT / 8;
        float sc[NK][4];
#pragma unroll
        for (int n = 0; n < NK; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        if constexpr (BF) {
          const int key = ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int n = 0; n < NK; n += 2) {
              uint32_t b[4];
              ldsm4(kb + (8 * n + key) * RB + (((2 * kk + ((lane >> 3) & 1)) ^ (key & 7)) << 4), b);
              mma_bf16(sc[n], qh[kk], b[0], b[1]);
              mma_bf16(sc[n + 1], qh[kk], b[2], b[3]);
            }
          }
#pragma unroll
          for (int n = 0; n < NK; ++n) {  // q_hi k + q_lo k
            sc[n][0] = add_low(sc[n][0], sc[n][2]);
            sc[n][1] = add_low(sc[n][1], sc[n][3]);
          }
        } else {
          // The tensor cores drop bits when they add to a running sum: the small products and
          // every fourth of the large ones have a sum of their own, added up in fp32.
          float sl[4] = {0.f, 0.f, 0.f, 0.f}, sh[4][4];
#pragma unroll
          for (int e = 0; e < 16; ++e) sh[e >> 2][e & 3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            uint32_t h0, l0, h1, l1;
            const uint32_t rowa = kb + gr * RB + t4 * 4;
            split_tf32(lds32(rowa + (((2 * kk) ^ gr) << 4)), h0, l0);
            split_tf32(lds32(rowa + (((2 * kk + 1) ^ gr) << 4)), h1, l1);
            mma_tf32(sl, ql[kk], h0, h1);
            mma_tf32(sl, qh[kk], l0, l1);
            mma_tf32(sh[kk & 3], qh[kk], h0, h1);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[0][e] = add_low((sh[0][e] + sh[1][e]) + (sh[2][e] + sh[3][e]), sl[e]);
        }
        if (!full) {
#pragma unroll
          for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int e = 0; e < 2 * HR; ++e) {
              const int key = k0 + n * 8 + 2 * t4 + (e & 1);
              const int lim = ctx ? cu.q.C - 1 : min(vis[e >> 1], cu.q.L - 1);
              if (key > lim) sc[n][e] = -INFINITY;
            }
        }
        float alpha[HR];
#pragma unroll
        for (int hf = 0; hf < HR; ++hf) {
          float mx = fmaxf(sc[0][2 * hf], sc[0][2 * hf + 1]);
#pragma unroll
          for (int n = 1; n < NK; ++n) mx = fmaxf(mx, fmaxf(sc[n][2 * hf], sc[n][2 * hf + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[hf], mx * p.scale_log2);
          const float use = mn == -INFINITY ? 0.f : mn;
          alpha[hf] = ex2(m[hf] - use);  // 0 while nothing has been seen
          m[hf] = mn;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int e = 2 * hf; e < 2 * hf + 2; ++e) {
              sc[n][e] = ex2(fmaf(sc[n][e], p.scale_log2, -use));
              sum += sc[n][e];
            }
          l[hf] = fmaf(l[hf], alpha[hf], sum);
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[HR - 1] != 1.f)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[nt][0] *= alpha[0];
            o[nt][1] *= alpha[0];
            o[nt][2] *= alpha[HR - 1];
            o[nt][3] *= alpha[HR - 1];
          }
        }
        if constexpr (BF) {
          const int key = lane & 15;
#pragma unroll
          for (int n = 0; n < NK; n += 2) {
            uint32_t a[4];  // rows 0-7 high parts, 8-15 low parts
            split_bf16(sc[n][0], sc[n][1], a[0], a[1]);
            split_bf16(sc[n + 1][0], sc[n + 1][1], a[2], a[3]);
#pragma unroll
            for (int nn = 0; nn < NT / 2; ++nn) {
              uint32_t b[4];
              ldsm4t(vb + (8 * n + key) * RB + (((2 * nn + (lane >> 4)) ^ (key & 7)) << 4), b);
              mma_bf16(o[2 * nn], a, b[0], b[1]);
              mma_bf16(o[2 * nn + 1], a, b[2], b[3]);
            }
          }
        } else {
          // key order of the k index: t4 -> key 2 t4, t4 + 4 -> key 2 t4 + 1, so that the
          // score fragment is the probability fragment
          uint32_t ah[4], al[4];
          split_tf32(sc[0][0], ah[0], al[0]);
          split_tf32(sc[0][2], ah[1], al[1]);
          split_tf32(sc[0][1], ah[2], al[2]);
          split_tf32(sc[0][3], ah[3], al[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t h0, l0, h1, l1;
            const uint32_t ch = 2 * nt + (gr >> 2), in = (gr & 3) * 4;
            split_tf32(lds32(vb + (2 * t4) * RB + ((ch ^ (2 * t4)) << 4) + in), h0, l0);
            split_tf32(lds32(vb + (2 * t4 + 1) * RB + ((ch ^ (2 * t4 + 1)) << 4) + in), h1, l1);
            // (added to the running sum in fp32)
            float dl[4] = {0.f, 0.f, 0.f, 0.f}, dh[4] = {0.f, 0.f, 0.f, 0.f};
            mma_tf32(dl, al, h0, h1);
            mma_tf32(dl, ah, l0, l1);
            mma_tf32(dh, ah, h0, h1);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][e] += add_low(dh[e], dl[e]);
          }
        }
      }

      // ---- the block's rows, or this range's partial of them
      if constexpr (BF) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {  // p_hi v + p_lo v
          o[nt][0] = add_low(o[nt][0], o[nt][2]);
          o[nt][1] = add_low(o[nt][1], o[nt][3]);
        }
      }
#pragma unroll
      for (int hf = 0; hf < HR; ++hf) {
        l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
        l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
        const int lr = gr + 8 * hf;
        if (lr >= nrow) continue;
        if (begins && ends) {
          const int row = cu.blk * kRows + lr;
          const int tok = row / Gq, hq = head * Gq + row % Gq;
          const float inv = l[hf] > 0.f ? 1.f / l[hf] : 0.f;
          T* out = static_cast<T*>(p.O) + ((int64_t)(cu.q.a + tok) * p.h_q + hq) * D + 2 * t4;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (BF)
              *reinterpret_cast<uint32_t*>(out + 8 * nt) =
                  pack_bf16(o[nt][2 * hf] * inv, o[nt][2 * hf + 1] * inv);
            else
              *reinterpret_cast<float2*>(out + 8 * nt) =
                  make_float2(o[nt][2 * hf] * inv, o[nt][2 * hf + 1] * inv);
          }
        } else {
          const int64_t slot =
              (((int64_t)s * 2 + (begins ? 1 : 0)) * p.h_kv + head) * kRows + lr;
          float* out = p.part_o + slot * D + 2 * t4;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            *reinterpret_cast<float2*>(out + 8 * nt) = make_float2(o[nt][2 * hf], o[nt][2 * hf + 1]);
          if (t4 == 0)
            *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(m[hf], l[hf]);
        }
      }
      if (begins && !ends) {  // the range's last item: it goes on in the next ranges
        const int64_t end = pre[cu.r] + (int64_t)(cu.blk + 1) * cu.TPP - 1;
        tail = make_int4(cu.q.a, cu.q.T, cu.blk, range_of(end, total, S));
      }
      if (ends && v < n_tiles) {
        cu.t = cu.TPP - 1;
        step(cu);
      }
    }
    cp_wait<0>();
  }
  if (head == 0 && lane == 0 && s < S_max) p.tail[s] = tail;
  if constexpr (BF)
    if (p.tc_rows != INT_MAX) rotate_queries<D>(p, w_all, gridDim.x * kWarps, lane,
                        reinterpret_cast<float2*>(sm_raw + kWarps * kRing + warp * kAngles), turns);
  if (err) cta_err = err;
  __syncthreads();
  if (tid == 0) p.err_cta[blockIdx.x] = cta_err;
}

// Partials of the query blocks that no single range held whole: the block that range s begins
// and the ranges s + 1 .. tail.w go on with, out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i
// over its segments i in a fixed order. One wave of CTAs: each lists the blocks to fold (of both
// attention kernels, in the same order in every CTA), then the rows of blocks of few segments are
// dealt to single warps and those of many segments to whole CTAs (one request split over the
// machine has few rows of many segments). Few bytes: latency-bound.
constexpr int kFewSegments = 16;
constexpr int kQuad = 4;          // rows of a tcgen05 block that a warp folds together
constexpr int kMaxTails = 2048;   // ranges of both kernels
template <int EL> struct Fold {   // a lane holds EL consecutive elements of the row
  static constexpr int U = 8;
  float M = -INFINITY, L = 0.f, acc[EL];
  __device__ __forceinline__ Fold() {
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] = 0.f;
  }
  static __device__ __forceinline__ void load(float (&v)[EL], const float* at) {
    if constexpr (EL == 4) {
      const float4 x = *reinterpret_cast<const float4*>(at);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(at);
      v[0] = x.x; v[1] = x.y;
    }
  }
  // segments i, i + step, i + 2 step, .. < n, U loads in flight; slot(i): the row's partial
  template <typename F>
  __device__ __forceinline__ void run(int i, int step, int n, const float* ml, const float* o,
                                      int lane, F slot) {
#pragma unroll 1
    for (; i < n; i += step * U) {
      float2 ml2[U];
      float ov[U][EL];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = i + u * step;
        ml2[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < EL; ++e) ov[u][e] = 0.f;
        if (j < n) {
          const int64_t at = slot(j);
          ml2[u] = *reinterpret_cast<const float2*>(ml + at * 2);
          load(ov[u], o + at * (EL * 32) + lane * EL);
        }
      }
      float Mn = M;
#pragma unroll
      for (int u = 0; u < U; ++u) Mn = fmaxf(Mn, ml2[u].x);
      rescale(Mn);
      const float use = Mn == -INFINITY ? 0.f : Mn;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = ex2(ml2[u].x - use);
        L = fmaf(ml2[u].y, w, L);
#pragma unroll
        for (int e = 0; e < EL; ++e) acc[e] = fmaf(ov[u][e], w, acc[e]);
      }
    }
  }
  __device__ __forceinline__ void add2(float2 a, const float (&oa)[EL], float2 b,
                                       const float (&ob)[EL]) {
    const float Mn = fmaxf(M, fmaxf(a.x, b.x));
    rescale(Mn);
    const float use = Mn == -INFINITY ? 0.f : Mn;
    const float wa = ex2(a.x - use), wb = ex2(b.x - use);
    L = fmaf(b.y, wb, fmaf(a.y, wa, L));
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] = fmaf(ob[e], wb, fmaf(oa[e], wa, acc[e]));
  }
  __device__ __forceinline__ void rescale(float Mn) {
    const float a = ex2(M - (Mn == -INFINITY ? 0.f : Mn));
    L *= a;
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] *= a;
    M = Mn;
  }
  template <typename T> __device__ __forceinline__ void store(T* row, int lane) const {
    const float inv = L > 0.f ? 1.f / L : 0.f;
    T* out = row + lane * EL;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int e = 0; e < EL; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    } else {
#pragma unroll
      for (int e = 0; e < EL; e += 2)
        *reinterpret_cast<float2*>(out + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
    }
  }
};
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads, 3) paged_merge_kernel(PagedAttendParams p, int S,
                                                                       int tc_grid, int n_cta) {
  constexpr int EL = D / 32;  // elements a lane holds
  constexpr int W = kMergeThreads / 32;
  constexpr int kRows = kBlockRows<T>;
  __shared__ float sh_o[W][D];
  __shared__ float sh_m[W], sh_l[W];
  // blocks of few and of many segments: which range, first row task, how many rows
  __shared__ int16_t item[2][kMaxTails];
  __shared__ int32_t start[2][kMaxTails + 1];
  __shared__ unsigned long long warp_tot[W];
  __shared__ int code;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Gq = p.h_q / p.h_kv, TB = 256 / Gq;
  if (tid == 0) code = 0;
  wait_then_let_start();
  if (blockIdx.x == 0)  // the call's status word
    for (int i = tid; i < n_cta; i += kMergeThreads)
      if (p.err_cta[i]) code = p.err_cta[i];
  auto tail_of = [&](int i) { return i < S ? p.tail[i] : p.tc_tail[2 * (i - S)]; };
  int n_item[2] = {0, 0}, n_task[2] = {0, 0};
#pragma unroll 1
  for (int i0 = 0; i0 < S + tc_grid; i0 += kMergeThreads) {
    const int i = i0 + tid;
    int tasks = 0, many = 0;
    if (i < S + tc_grid) {
      const int4 t = tail_of(i);
      if (t.x >= 0) {
        many = t.w - (i < S ? i : i - S) + 1 > kFewSegments;
        tasks = i < S ? min(kRows, t.y * Gq - t.z * kRows) * p.h_kv
                      : min(TB, t.y - t.z * TB) * Gq;
        if (i >= S && !many) tasks = (tasks + kQuad - 1) / kQuad;
      }
    }
    // one scan of the tasks of both lists (32 bits each), ballots for the items
    unsigned long long inc = (unsigned long long)tasks << (many ? 32 : 0);
    const unsigned long long own = inc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned few_m = __ballot_sync(0xffffffffu, tasks > 0 && !many);
    const unsigned many_m = __ballot_sync(0xffffffffu, tasks > 0 && many);
    __shared__ int warp_items[W];
    if (lane == 31) warp_tot[warp] = inc;
    if (lane == 0) warp_items[warp] = __popc(few_m) | __popc(many_m) << 16;
    __syncthreads();
    unsigned long long before = 0, all = 0;
    int items_before = 0, items_all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) {
        before += warp_tot[w];
        items_before += warp_items[w];
      }
      all += warp_tot[w];
      items_all += warp_items[w];
    }
    if (tasks > 0) {
      const unsigned m = (many ? many_m : few_m) & ((1u << lane) - 1u);
      const int at = n_item[many] + ((items_before >> (many * 16)) & 0xffff) + __popc(m);
      item[many][at] = (int16_t)i;
      start[many][at] = n_task[many] + (int)((before + inc - own) >> (many * 32));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      n_item[k] += (items_all >> (k * 16)) & 0xffff;
      n_task[k] += (int)(all >> (k * 32));
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) {
    *p.err = code;
    if (code) set_err(p.step_err, code);
  }
  // row task t of list k: where its partials and its row of O are
  struct Row {
    const float* ml;
    const float* o;
    int64_t slot0, slot1, step;  // partial of segment 0, of segment 1, between later ones
    int n_seg, g0;               // g0: first row's query head of the group (tcgen05 blocks)
    T* out;
  };
  auto locate = [&](int k, int t, int* n_row) {
    int lo = 0, hi = n_item[k];
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[k][mid] <= t) lo = mid;
      else hi = mid;
    }
    const int i = item[k][lo];
    int x = t - start[k][lo];
    const int4 tail = tail_of(i);
    *n_row = 1;
    Row r;
    int tok, hq;
    if (i < S) {
      const int nrow = min(kRows, tail.y * Gq - tail.z * kRows);
      const int head = x / nrow, lr = x % nrow, row = tail.z * kRows + lr;
      r.ml = p.part_ml;
      r.o = p.part_o;
      r.step = (int64_t)2 * p.h_kv * kRows;
      r.slot0 = i * r.step + (int64_t)(p.h_kv + head) * kRows + lr;  // the tail slot of i,
      r.slot1 = (i + 1) * r.step + (int64_t)head * kRows + lr;       // then the head slots
      r.n_seg = tail.w - i + 1;
      tok = row / Gq;
      hq = head * Gq + row % Gq;
    } else {
      const int s = i - S;
      if (k == 0) {  // rows x .. x + n_row of the block
        x *= kQuad;
        *n_row = min(kQuad, min(TB, tail.y - tail.z * TB) * Gq - x);
        r.g0 = x % Gq;
      }
      r.ml = p.tc_ml;
      r.o = p.tc_o;
      r.step = 512;
      r.slot0 = (int64_t)s * 512 + 256 + x;
      r.slot1 = (int64_t)(s + 1) * 512 + x;
      r.n_seg = tail.w - s + 1;
      tok = tail.z * TB + x / Gq;
      hq = p.tc_tail[2 * s + 1].x * Gq + x % Gq;
    }
    r.out = static_cast<T*>(p.O) + ((int64_t)(tail.x + tok) * p.h_q + hq) * D;
    return r;
  };
#pragma unroll 1
  for (int t = blockIdx.x * W + warp; t < n_task[0]; t += gridDim.x * W) {
    int n_row;
    const Row r = locate(0, t, &n_row);
    auto slot = [&](int i) { return i == 0 ? r.slot0 : r.slot1 + (i - 1) * r.step; };
    if (r.ml != p.tc_ml) {
      Fold<EL> f;
      f.run(0, 1, r.n_seg, r.ml, r.o, lane, slot);
      f.store(r.out, lane);
      continue;
    }
    Fold<EL> f[kQuad];  // kQuad rows a segment at a time, two segments' loads in flight
#pragma unroll 1
    for (int i = 0; i < r.n_seg; i += 2) {
      float2 ml2[2][kQuad];
      float ov[2][kQuad][EL];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < kQuad; ++q) {
          ml2[u][q] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int e = 0; e < EL; ++e) ov[u][q][e] = 0.f;
          if (i + u < r.n_seg && q < n_row) {
            const int64_t at = slot(i + u) + q;
            ml2[u][q] = *reinterpret_cast<const float2*>(r.ml + at * 2);
            Fold<EL>::load(ov[u][q], r.o + at * D + lane * EL);
          }
        }
#pragma unroll
      for (int q = 0; q < kQuad; ++q) f[q].add2(ml2[0][q], ov[0][q], ml2[1][q], ov[1][q]);
    }
    T* out = r.out;
#pragma unroll
    for (int q = 0; q < kQuad; ++q) {
      if (q < n_row) f[q].store(out, lane);
      // the next row: the group's next query head, or the next token's first one
      out += (r.g0 + q + 1) % Gq == 0 ? (int64_t)(p.h_q - Gq + 1) * D : D;
    }
  }
#pragma unroll 1
  for (int t = blockIdx.x; t < n_task[1]; t += gridDim.x) {
    int n_row;
    const Row r = locate(1, t, &n_row);
    Fold<EL> f;
    f.run(warp, W, r.n_seg, r.ml, r.o, lane,
          [&](int i) { return i == 0 ? r.slot0 : r.slot1 + (i - 1) * r.step; });
#pragma unroll
    for (int e = 0; e < EL; ++e) sh_o[warp][e * 32 + lane] = f.acc[e];
    if (lane == 0) {
      sh_m[warp] = f.M;
      sh_l[warp] = f.L;
    }
    __syncthreads();
    if (warp == 0) {
      float Mn = f.M;
      for (int u = 1; u < W; ++u) Mn = fmaxf(Mn, sh_m[u]);
      f.rescale(Mn);
      const float use = Mn == -INFINITY ? 0.f : Mn;
      for (int u = 1; u < W; ++u) {
        const float w = ex2(sh_m[u] - use);
        f.L = fmaf(sh_l[u], w, f.L);
#pragma unroll
        for (int e = 0; e < EL; ++e) f.acc[e] = fmaf(sh_o[u][e * 32 + lane], w, f.acc[e]);
      }
      f.store(r.out, lane);
    }
    __syncthreads();  // the shared rows are written anew
  }
}

template <typename T, int D>
cudaError_t launch(const PagedAttendParams& p, const PagedPlan& pl, cudaStream_t st) {
  auto kfn = paged_attend_kernel<T, D>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = allow_smem_once(reinterpret_cast<const void*>(kfn), kMaxSmem, ready);
  if (e != cudaSuccess) return e;
  e = launch_early(kfn, dim3(pl.grid), dim3(kThreads), pl.smem, st, p, pl.S);
  if (e != cudaSuccess) return e;
  if constexpr (sizeof(T) == 2) {  // its CTAs start as the warp-level kernel's end
    if (pl.tc_grid > 0) e = launch_paged_attend_tc(p, pl.tc_grid, D, st);
    if (e != cudaSuccess) return e;
  }
  // the merge kernel is launched while the attention runs and waits for it on the device
  return launch_early(paged_merge_kernel<T, D>, dim3(pl.grid * 3), dim3(kMergeThreads), 0, st, p,
                      pl.S, pl.tc_grid, pl.grid + pl.tc_grid);  // one wave
}

}  // namespace pga

PagedPlan paged_attend_plan(int n_rows, int n_req, int h_q, int h_kv, int d, int dtype, int sms) {
  PagedPlan pl{};
  auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
  // one CTA per SM; more when the heads alone need more warps
  pl.grid = std::max(sms, (h_kv + pga::kWarps - 1) / pga::kWarps);
  // (the merge lists the ranges of both kernels in shared memory: 1,332 on a B200)
  pl.S = std::min(pl.grid * pga::kWarps / h_kv, pga::kMaxTails - sms);
  // The tcgen05 kernel serves the bf16 requests with more than 8 query rows per KV head: 16
  // requests of 8,000 rows (8 KV heads, d = 128) take 92 us on the warp-level kernel and 109 here
  // with 8 query rows each, 165 and 110 with 9, 289 and 111 with 32 (64 of 1,000 rows at d = 64
  // and 4 KV heads: 19 and 40 with 8, 27 and 40 with 12, 36 and 40 with 20). The
  // host sees only the totals: it leaves the launch out where no request can have so many, and
  // where there is at most one new token per slot of the table (a decode step, where the launch
  // finds nothing and costs 4 to 5 us: the 64 requests with 8 rows each, 19.4 -> 24.7 us). What
  // that costs: a chunk in a step of no more rows than slots stays on the warp-level kernel, which
  // passes over the keys for every 8 rows (one request over 32,768 rows in a table of 256 slots:
  // 4 tokens 41 us against 51, 16 tokens 118 against 53, 200 tokens 1,260 against 157).
  const int Gq = h_q / h_kv;
  const bool tc = dtype == 1 && Gq <= 256 && (int64_t)n_rows * Gq > kPagedWarpRows &&
                  (n_rows > n_req || Gq > kPagedWarpRows);
  pl.tc_grid = tc ? sms : 0;
  const size_t slots = (size_t)pl.S * 2 * h_kv * (dtype == 1 ? kPagedWarpRows : 16);
  pl.err_bytes = al((size_t)(pl.grid + pl.tc_grid) * sizeof(int));
  pl.tail_bytes = al((size_t)pl.S * sizeof(int4));
  pl.ml_bytes = al(slots * 2 * sizeof(float));
  pl.o_bytes = al(slots * d * sizeof(float));
  pl.tc_tail_bytes = al((size_t)pl.tc_grid * 2 * sizeof(int4));
  pl.tc_ml_bytes = al((size_t)pl.tc_grid * 2 * 256 * 2 * sizeof(float));
  pl.tc_o_bytes = al((size_t)pl.tc_grid * 2 * 256 * d * sizeof(float));
  pl.q_bytes = tc ? al((size_t)n_rows * h_q * d * 2 * 2) : 0;
  pl.smem = pga::kWarps * (pga::kRing + pga::kAngles) +
            (n_req <= pga::kReqCache
                 ? (pga::kReqCache + 4) * sizeof(int32_t) + pga::kReqCache * sizeof(int4)
                 : ((size_t)n_req + 1) * sizeof(int32_t));
  return pl;
}

cudaError_t launch_paged_attend(const PagedAttendParams& p, const PagedPlan& pl, int dtype, int d,
                                cudaStream_t st) {
  if (dtype == 1)
    return d == 128 ? pga::launch<__nv_bfloat16, 128>(p, pl, st)
                    : pga::launch<__nv_bfloat16, 64>(p, pl, st);
  return d == 128 ? pga::launch<float, 128>(p, pl, st) : pga::launch<float, 64>(p, pl, st);
}

}  // namespace msa
