// paged_attend.cu - attention of ragged requests over [routed memory ; paged local context]: the
// operation of sparse generation
//   [news.neo-ai.one article, "グローバル RoPE（アクティブコンテキスト）" and "推論パイプライン";
//    ruixiangma.github.io blog, "三阶段推理流程"]
// for a batch whose requests differ in length, with their local K/V in pages of one pool. Token i
// of request r's T new ones sits at local row j = len - T + i; its query, rotated at pos0 + j,
// attends over the request's memory rows and its local rows <= j (keys stored rotated):
//   O = softmax(scale q . k) v, 0 where nothing is visible.
//
// The kernel of this file streams each key row once per 16 query rows and is the one for few
// query rows per KV head (single tokens) and for fp32. A warp works alone: for one KV head it
// takes a contiguous range of the flattened list (request, block of 16 query rows, tile of
// keys), copies the tiles with cp.async into its own ring in shared memory (no barrier between
// warps), forms the scores and P V with warp-level MMAs (bf16; fp32 as three tf32 products of
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
constexpr int kRows = kPagedWarpRows;  // query rows of a block (the MMA's M)
constexpr int kRing = 24576;        // bytes of a warp's ring
constexpr int kMinTiles = 4;        // a range is at least this many tiles
constexpr int kMergeThreads = 256;

template <typename T, int D> struct Geo {
  static constexpr int KT = sizeof(T) == 2 ? 16 : 8;      // keys of a tile
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
// x = hi + lo with both in tf32 (11 significant bits each): hi hi + hi lo + lo hi leaves out
// lo lo, 2^-22 of the product, next to fp32's own 2^-24
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  const float rest = x - __uint_as_float(hi);
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(rest));
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
// another, 16-byte chunk c of a row at c ^ (row within its block & 7). A warp takes a token: lane =
// one 16-byte chunk of the lower half of a head and its partner half a head on.
template <int D>
__device__ __forceinline__ void rotate_queries(const PagedAttendParams& p, int w, int n_warps,
                                               int lane) {
  constexpr int HC = D / 16;       // chunks of half a head
  constexpr int HPW = 32 / HC;     // heads a warp takes at once
  const int Gq = p.h_q / p.h_kv, TB = 256 / Gq;
  const int c = lane % HC;
  unsigned long long F[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) F[e] = p.rope_turns[c * 8 + e];
  const int64_t rows = (int64_t)p.n_rows * Gq;
  for (int i = w; i < p.n_rows; i += n_warps) {
    int lo = 0, hi = p.n_req;      // the request of token i: row_start[lo] <= i < row_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.row_start + mid) <= i) lo = mid;
      else hi = mid;
    }
    int ignore = 0;
    const PagedReq q = paged_req(p, lo, p.tc_rows, INT_MAX, &ignore);
    const int t = i - q.a;
    if (t < 0 || t >= q.T) continue;
    const int64_t pos = (int64_t)p.pos0 + q.L - q.T + t;
    float2 cs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = p.rope ? rot_turns(pos, F[e]) : make_float2(1.f, 0.f);
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.Q) + i * p.q_stride;
#pragma unroll 2
    for (int h = lane / HC; h < p.h_q; h += HPW) {
      using V = Vec<__nv_bfloat16, 8>;
      const uint4 ra = __ldg(reinterpret_cast<const uint4*>(src + h * D + c * 8));
      const uint4 rb = __ldg(reinterpret_cast<const uint4*>(src + h * D + c * 8 + D / 2));
      float a[8], b[8];
      V::unpack(ra, a);
      V::unpack(rb, b);
      uint32_t oa[4], ob[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 c0 = cs[2 * e], c1 = cs[2 * e + 1];
        oa[e] = pack_bf16(a[2 * e] * c0.x - b[2 * e] * c0.y,
                          a[2 * e + 1] * c1.x - b[2 * e + 1] * c1.y);
        ob[e] = pack_bf16(b[2 * e] * c0.x + a[2 * e] * c0.y,
                          b[2 * e + 1] * c1.x + a[2 * e + 1] * c1.y);
      }
      const int kv = h / Gq, g = h % Gq;
      const int x = ((t % TB) * Gq + g) & 7;
      const int64_t row = (int64_t)i * Gq + g;
      auto put = [&](int chunk, const uint32_t (&v)[4]) {  // chunk of the head's row
        __nv_bfloat16* dst = p.q_rot + (((int64_t)kv * (D / 64) + chunk / 8) * rows + row) * 64 +
                             (((chunk & 7) ^ x) << 3);
        *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
      };
      put(c, oa);
      put(c + HC, ob);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) paged_attend_kernel(PagedAttendParams p, int S_max) {
  using G = Geo<T, D>;
  constexpr int KT = G::KT, RB = G::RB, TILE = G::TILE, NST = G::NST;
  constexpr bool BF = sizeof(T) == 2;
  constexpr int NT = D / 8;                      // 8-wide output tiles
  constexpr int KS = BF ? D / 16 : D / 8;        // k steps of the scores
  extern __shared__ __align__(128) unsigned char sm_raw[];
  int64_t* pre = reinterpret_cast<int64_t*>(sm_raw + kWarps * kRing);  // [n_req + 1] first tile
  __shared__ int64_t warp_tot[kWarps];
  __shared__ int cta_err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Gq = p.h_q / p.h_kv;

  // the dependent merge kernel may be set up while this one runs (it waits for the results)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
    if (r < p.n_req) pre[r] = base + inc - v;
    __syncthreads();
  }
  if (tid == 0) pre[p.n_req] = carry;
  __syncthreads();
  const int64_t total = carry;
  const int S = (int)max((int64_t)1, min((int64_t)S_max, total / kMinTiles));
  const int w_all = blockIdx.x * kWarps + warp;
  const int s = w_all / p.h_kv, head = w_all % p.h_kv;
  const int64_t x0 = s < S ? range_start(total, s, S) : total;
  const int64_t x1 = s < S ? range_start(total, s + 1, S) : total;
  const int n_tiles = (int)(x1 - x0);
  int4 tail = make_int4(-1, 0, 0, 0);

  if (n_tiles > 0) {
    const uint32_t ring = smem_u32(sm_raw) + warp * kRing;
    const int n_slot_pages = p.n_pages;
    // where a tile of the list lies
    struct Cur {
      int r, blk, t, TPP, CT, nb;
      PagedReq q;
    };
    auto enter = [&](Cur& c, int r) {  // request r's geometry (r has tiles)
      int ignore = 0;
      c.r = r;
      c.q = paged_req(p, r, 0, p.tc_rows, &ignore);
      c.CT = ctx_tiles<KT>(c.q);
      c.TPP = block_tiles<KT>(c.q);
      c.nb = (int)(((long long)c.q.T * Gq + kRows - 1) / kRows);
    };
    auto step = [&](Cur& c) {  // the next tile of the list (only called when there is one)
      if (++c.t < c.TPP) return;
      c.t = 0;
      if (++c.blk < c.nb) return;
      c.blk = 0;
      int r = c.r + 1;
      while (pre[r + 1] == pre[r]) ++r;
      enter(c, r);
    };
    // last local row that the block's last token sees
    auto block_last = [&](const Cur& c) {
      const int t_last = min((c.blk * kRows + kRows - 1) / Gq, c.q.T - 1);
      return c.q.L - c.q.T + t_last;
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
      const int64_t off = x0 - pre[lo];
      ld.blk = (int)(off / ld.TPP);
      ld.t = (int)(off % ld.TPP);
    }
    Cur cu = ld;  // the tile being computed; ld is the tile being loaded

    // a tile's page is looked up one tile before its copies go out
    auto lookup = [&](const Cur& c) -> int {
      if (c.t < c.CT) return 0;
      const int k0 = (c.t - c.CT) * KT;
      if (k0 >= c.q.L || k0 > block_last(c)) return -1;  // nothing of it is seen
      return __ldg(p.table + (int64_t)c.r * p.max_pages + (k0 >> p.page_shift));
    };
    int page = lookup(ld);
    auto issue = [&](int v) {  // copies of tile v of the range into stage v % NST
      const Cur& c = ld;
      const uint32_t st = ring + (uint32_t)(v % NST) * (2 * TILE);
      const T* ks = nullptr;
      const T* vs = nullptr;
      int valid = 0;
      if (c.t < c.CT) {
        const int64_t at = ((int64_t)c.r * p.max_ctx + c.t * KT) * p.h_kv + head;
        ks = static_cast<const T*>(p.cK) + at * D;
        vs = static_cast<const T*>(p.cV) + at * D;
        valid = min(KT, c.q.C - c.t * KT);
      } else {
        const int k0 = (c.t - c.CT) * KT;
        if (k0 < c.q.L && k0 <= block_last(c)) {
          if (page < 0 || page >= n_slot_pages) {
            err = kErrBadIndex;
          } else {
            const int64_t row = ((int64_t)page << p.page_shift) +
                                (k0 & ((1 << p.page_shift) - 1));
            ks = static_cast<const T*>(p.K_pages) + (row * p.h_kv + head) * D;
            vs = static_cast<const T*>(p.V_pages) + (row * p.h_kv + head) * D;
            valid = min(KT, c.q.L - k0);
          }
        }
      }
      if (ks != nullptr) {  // rows past the end are filled with zeros (their V meets P = 0)
        constexpr int CPR = RB / 16;      // 16-byte chunks of a row
        constexpr int RPI = 32 / CPR;     // rows a warp instruction copies
        const int c16 = lane % CPR, r0 = lane / CPR;
        const int64_t pitch = (int64_t)p.h_kv * RB;
#pragma unroll
        for (int i = 0; i < KT / RPI; ++i) {
          const int row = r0 + i * RPI;
          const bool ok = row < valid;
          const int64_t off = ok ? row * pitch + c16 * 16 : 0;
          const uint32_t dst = st + row * RB + ((c16 ^ (row & 7)) << 4);
          cp16_zfill(dst, reinterpret_cast<const char*>(ks) + off, ok);
          cp16_zfill(dst + TILE, reinterpret_cast<const char*>(vs) + off, ok);
        }
      }
      if (v + 1 < n_tiles) {
        step(ld);
        page = lookup(ld);
      }
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
    float m[2], l[2];
    int v = 0;
    while (v < n_tiles) {
      // ---- one query block's share of the range
      const bool begins = cu.t == 0;
      const int t_end = (int)min((int64_t)cu.TPP, (int64_t)cu.t + (n_tiles - v));
      const bool ends = t_end == cu.TPP;
      const int nrow = min(kRows, (int)min((long long)kRows, (long long)cu.q.T * Gq - (long long)cu.blk * kRows));
      int vis[2];  // last local row that query rows gr and gr + 8 see
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int row = cu.blk * kRows + min(gr + 8 * hf, nrow - 1);
        const int tok = row / Gq, hq = head * Gq + row % Gq;
        const int j = cu.q.L - cu.q.T + tok;
        vis[hf] = j;
        const T* src = static_cast<const T*>(p.Q) + (int64_t)(cu.q.a + tok) * p.q_stride + hq * D;
        const int64_t pos = (int64_t)p.pos0 + j;
        // a lane's fragment elements of dims i and i + D/2 are its own: it rotates them itself
        if constexpr (BF) {
#pragma unroll
          for (int kk = 0; kk < KS / 2; ++kk) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = kk * 16 + e * 8 + 2 * t4;
              const uint32_t lo = __ldg(reinterpret_cast<const uint32_t*>(src + i));
              const uint32_t hi = __ldg(reinterpret_cast<const uint32_t*>(src + i + D / 2));
              float2 c0 = make_float2(1.f, 0.f), c1 = c0;
              if (p.rope) {
                c0 = rot_turns(pos, p.rope_turns[i]);
                c1 = rot_turns(pos, p.rope_turns[i + 1]);
              }
              const float a0 = __uint_as_float(lo << 16), a1 = __uint_as_float(lo & 0xFFFF0000u);
              const float b0 = __uint_as_float(hi << 16), b1 = __uint_as_float(hi & 0xFFFF0000u);
              // rounded to bf16 for the tensor cores, as the keys were when appended
              qh[kk][hf + 2 * e] = pack_bf16(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
              qh[kk + KS / 2][hf + 2 * e] =
                  pack_bf16(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < KS / 2; ++kk) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = kk * 8 + e * 4 + t4;
              const float a0 = __ldg(reinterpret_cast<const float*>(src) + i);
              const float b0 = __ldg(reinterpret_cast<const float*>(src) + i + D / 2);
              const float2 c0 = p.rope ? rot_turns(pos, p.rope_turns[i]) : make_float2(1.f, 0.f);
              split_tf32(a0 * c0.x - b0 * c0.y, qh[kk][hf + 2 * e], ql[kk][hf + 2 * e]);
              split_tf32(b0 * c0.x + a0 * c0.y, qh[kk + KS / 2][hf + 2 * e],
                         ql[kk + KS / 2][hf + 2 * e]);
            }
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
      const int first_vis = cu.q.L - cu.q.T + cu.blk * kRows / Gq;  // of the block's first token
      const int last_vis = block_last(cu);

      for (; cu.t < t_end; ++cu.t, ++v) {
        cp_wait<NST - 2>();
        __syncwarp();
        if (v + NST - 1 < n_tiles) issue(v + NST - 1);
        cp_commit();
        const bool ctx = cu.t < cu.CT;
        const int k0 = ctx ? cu.t * KT : (cu.t - cu.CT) * KT;
        if (!ctx && (k0 >= cu.q.L || k0 > last_vis)) continue;  // nothing visible
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
            uint32_t b[4];
            ldsm4(kb + key * RB + (((2 * kk + ((lane >> 3) & 1)) ^ (key & 7)) << 4), b);
            mma_bf16(sc[0], qh[kk], b[0], b[1]);
            mma_bf16(sc[1], qh[kk], b[2], b[3]);
          }
        } else {
          float sl[4] = {0.f, 0.f, 0.f, 0.f};  // the small products apart: two shorter chains
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            uint32_t h0, l0, h1, l1;
            const uint32_t rowa = kb + gr * RB + t4 * 4;
            split_tf32(lds32(rowa + (((2 * kk) ^ gr) << 4)), h0, l0);
            split_tf32(lds32(rowa + (((2 * kk + 1) ^ gr) << 4)), h1, l1);
            mma_tf32(sl, ql[kk], h0, h1);
            mma_tf32(sl, qh[kk], l0, l1);
            mma_tf32(sc[0], qh[kk], h0, h1);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[0][e] += sl[e];
        }
        if (!full) {
#pragma unroll
          for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = k0 + n * 8 + 2 * t4 + (e & 1);
              const int lim = ctx ? cu.q.C - 1 : min(vis[e >> 1], cu.q.L - 1);
              if (key > lim) sc[n][e] = -INFINITY;
            }
        }
        float alpha[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
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
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[nt][0] *= alpha[0];
            o[nt][1] *= alpha[0];
            o[nt][2] *= alpha[1];
            o[nt][3] *= alpha[1];
          }
        }
        if constexpr (BF) {
          // the probabilities enter the product in bf16 (their sum above in fp32)
          const uint32_t a[4] = {pack_bf16(sc[0][0], sc[0][1]), pack_bf16(sc[0][2], sc[0][3]),
                                 pack_bf16(sc[1][0], sc[1][1]), pack_bf16(sc[1][2], sc[1][3])};
          const int key = lane & 15;
#pragma unroll
          for (int nn = 0; nn < NT / 2; ++nn) {
            uint32_t b[4];
            ldsm4t(vb + key * RB + (((2 * nn + (lane >> 4)) ^ (key & 7)) << 4), b);
            mma_bf16(o[2 * nn], a, b[0], b[1]);
            mma_bf16(o[2 * nn + 1], a, b[2], b[3]);
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
            mma_tf32(o[nt], al, h0, h1);
            mma_tf32(o[nt], ah, l0, l1);
            mma_tf32(o[nt], ah, h0, h1);
          }
        }
      }

      // ---- the block's rows, or this range's partial of them
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
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
    if (p.tc_rows != INT_MAX) rotate_queries<D>(p, w_all, gridDim.x * kWarps, lane);
  if (err) cta_err = err;
  __syncthreads();
  if (tid == 0) p.err_cta[blockIdx.x] = cta_err;
}

// Partials of the query blocks that no single range held whole: the block that range s begins
// and the ranges s + 1 .. tail.w go on with, out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i
// over its segments i in a fixed order. The first S * h_kv CTAs take the warp-level kernel's
// blocks of 16 rows (a row's segments shared among the warps), kTcParts CTAs a range the tcgen05
// kernel's blocks of up to 256 rows (a warp a row). Few bytes: latency-bound.
template <int EL> struct Fold {
  float M = -INFINITY, L = 0.f, acc[EL];
  __device__ __forceinline__ Fold() {
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] = 0.f;
  }
  // segments i, i + step, i + 2 step, .. < n, four loads in flight; slot(i): the row's partial
  template <typename F>
  __device__ __forceinline__ void run(int i, int step, int n, const float* ml, const float* o,
                                      int lane, F slot) {
    for (; i < n; i += step * 4) {
      float mi[4], li[4], ov[4][EL];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = i + u * step;
        mi[u] = -INFINITY;
        li[u] = 0.f;
#pragma unroll
        for (int e = 0; e < EL; ++e) ov[u][e] = 0.f;
        if (j < n) {
          const int64_t at = slot(j);
          mi[u] = ml[at * 2];
          li[u] = ml[at * 2 + 1];
#pragma unroll
          for (int e = 0; e < EL; ++e) ov[u][e] = o[at * (EL * 32) + e * 32 + lane];
        }
      }
      float Mn = M;
#pragma unroll
      for (int u = 0; u < 4; ++u) Mn = fmaxf(Mn, mi[u]);
      rescale(Mn);
      const float use = Mn == -INFINITY ? 0.f : Mn;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float w = ex2(mi[u] - use);
        L = fmaf(li[u], w, L);
#pragma unroll
        for (int e = 0; e < EL; ++e) acc[e] = fmaf(ov[u][e], w, acc[e]);
      }
    }
  }
  __device__ __forceinline__ void rescale(float Mn) {
    const float a = ex2(M - (Mn == -INFINITY ? 0.f : Mn));
    L *= a;
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] *= a;
    M = Mn;
  }
  template <typename T> __device__ __forceinline__ void store(T* out, int lane) const {
    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int e = 0; e < EL; ++e) out[e * 32 + lane] = Elem<T>::from_f(acc[e] * inv);
  }
};
constexpr int kTcParts = 32;  // CTAs per range of the tcgen05 kernel: 8 of its 256 rows each

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(PagedAttendParams p, int S,
                                                                    int n_cta) {
  constexpr int EL = D / 32;  // elements a lane holds
  constexpr int W = kMergeThreads / 32;
  __shared__ float sh_o[W][D];
  __shared__ float sh_m[W], sh_l[W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Gq = p.h_q / p.h_kv;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0) {  // the call's status word
    __shared__ int code;
    if (tid == 0) code = 0;
    __syncthreads();
    for (int i = tid; i < n_cta; i += kMergeThreads)
      if (p.err_cta[i]) code = p.err_cta[i];
    __syncthreads();
    if (tid == 0) *p.err = code;
  }
  const int n_warp_level = S * p.h_kv;
  if ((int)blockIdx.x >= n_warp_level) {
    const int s = ((int)blockIdx.x - n_warp_level) / kTcParts;
    const int row = ((int)blockIdx.x - n_warp_level) % kTcParts * W + warp;
    const int4 tail = p.tc_tail[2 * s];
    if (tail.x < 0) return;
    const int head = p.tc_tail[2 * s + 1].x;
    const int TB = 256 / Gq;
    if (row >= min(TB, tail.y - tail.z * TB) * Gq) return;
    Fold<EL> f;
    f.run(0, 1, tail.w - s + 1, p.tc_ml, p.tc_o, lane, [&](int i) {
      return ((int64_t)(s + i) * 2 + (i == 0 ? 1 : 0)) * 256 + row;
    });
    const int tok = tail.z * TB + row / Gq, hq = head * Gq + row % Gq;
    f.store(static_cast<T*>(p.O) + ((int64_t)(tail.x + tok) * p.h_q + hq) * D, lane);
    return;
  }
  const int s = blockIdx.x / p.h_kv, head = blockIdx.x % p.h_kv;
  const int4 tail = p.tail[s];
  if (tail.x < 0) return;
  const int nrow = min(kRows, tail.y * Gq - tail.z * kRows);
  int wpr = 1;  // warps per row: a power of two, so that a row's warps are neighbours
  while (wpr * 2 * nrow <= W) wpr *= 2;
  const int g = warp % wpr;
  for (int r0 = 0; r0 < nrow; r0 += W / wpr) {
    const int lr = r0 + warp / wpr;
    const bool live = lr < nrow;
    Fold<EL> f;
    if (live)  // the tail slot of s, then the head slots
      f.run(g, wpr, tail.w - s + 1, p.part_ml, p.part_o, lane, [&](int i) {
        return (((int64_t)(s + i) * 2 + (i == 0 ? 1 : 0)) * p.h_kv + head) * kRows + lr;
      });
    if (wpr > 1) {
#pragma unroll
      for (int e = 0; e < EL; ++e) sh_o[warp][e * 32 + lane] = f.acc[e];
      if (lane == 0) {
        sh_m[warp] = f.M;
        sh_l[warp] = f.L;
      }
      __syncthreads();
      if (g == 0) {
        float Mn = f.M;
        for (int u = 1; u < wpr; ++u) Mn = fmaxf(Mn, sh_m[warp + u]);
        f.rescale(Mn);
        const float use = Mn == -INFINITY ? 0.f : Mn;
        for (int u = 1; u < wpr; ++u) {
          const float w = ex2(sh_m[warp + u] - use);
          f.L = fmaf(sh_l[warp + u], w, f.L);
#pragma unroll
          for (int e = 0; e < EL; ++e) f.acc[e] = fmaf(sh_o[warp + u][e * 32 + lane], w, f.acc[e]);
        }
      }
      __syncthreads();
    }
    if (live && g == 0) {
      const int row = tail.z * kRows + lr;
      const int tok = row / Gq, hq = head * Gq + row % Gq;
      f.store(static_cast<T*>(p.O) + ((int64_t)(tail.x + tok) * p.h_q + hq) * D, lane);
    }
  }
}

template <typename T, int D>
cudaError_t launch(const PagedAttendParams& p, const PagedPlan& pl, cudaStream_t st) {
  auto kfn = paged_attend_kernel<T, D>;
  cudaError_t e =
      cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)pl.smem);
  if (e != cudaSuccess) return e;
  kfn<<<pl.grid, kThreads, pl.smem, st>>>(p, pl.S);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if constexpr (sizeof(T) == 2) {  // its CTAs start as the warp-level kernel's end
    if (pl.tc_grid > 0) e = launch_paged_attend_tc(p, pl.tc_grid, D, st);
    if (e != cudaSuccess) return e;
  }
  // the merge kernel is launched while the attention runs and waits for it on the device
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(pl.S * p.h_kv + pl.tc_grid * kTcParts);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, D>, p, pl.S, pl.grid + pl.tc_grid);
}

}  // namespace pga

PagedPlan paged_attend_plan(int n_rows, int n_req, int h_q, int h_kv, int d, int dtype, int sms) {
  PagedPlan pl{};
  auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
  // one CTA per SM; more when the heads alone need more warps
  pl.grid = std::max(sms, (h_kv + pga::kWarps - 1) / pga::kWarps);
  pl.S = pl.grid * pga::kWarps / h_kv;
  // The tcgen05 kernel serves the bf16 requests with more than 16 query rows per KV head. The
  // host sees only the totals: it leaves the launch out where no request can have so many, and
  // where there is at most one new token per request on average (a decode step, where the launch
  // would cost its latency and find nothing; the warp-level kernel serves a longer request too).
  const int Gq = h_q / h_kv;
  const bool tc = dtype == 1 && Gq <= 256 && (int64_t)n_rows * Gq > kPagedWarpRows &&
                  n_rows > n_req;
  pl.tc_grid = tc ? sms : 0;
  const size_t slots = (size_t)pl.S * 2 * h_kv * pga::kRows;
  pl.err_bytes = al((size_t)(pl.grid + pl.tc_grid) * sizeof(int));
  pl.tail_bytes = al((size_t)pl.S * sizeof(int4));
  pl.ml_bytes = al(slots * 2 * sizeof(float));
  pl.o_bytes = al(slots * d * sizeof(float));
  pl.tc_tail_bytes = al((size_t)pl.tc_grid * 2 * sizeof(int4));
  pl.tc_ml_bytes = al((size_t)pl.tc_grid * 2 * 256 * 2 * sizeof(float));
  pl.tc_o_bytes = al((size_t)pl.tc_grid * 2 * 256 * d * sizeof(float));
  pl.q_bytes = tc ? al((size_t)n_rows * h_q * d * 2) : 0;
  pl.smem = pga::kWarps * pga::kRing + ((size_t)n_req + 1) * sizeof(int64_t);
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
