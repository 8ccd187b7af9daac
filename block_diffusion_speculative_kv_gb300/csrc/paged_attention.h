// Attention over a paged KV cache: parameters and work split shared by its
// kernels (paged_attention.cu).
#pragma once

#include <math_constants.h>

#include "mma_sync.cuh"
#include "paged.cuh"

namespace dfl {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLazy = 8.f;   // a row's reference maximum may lag by this much (base-2 units)

// Query heads per KV head, and division by them: the quotient by 2^32 / G rounded
// down is exact or one too small.
struct Heads {
  int G;
  uint32_t m;
  __device__ __forceinline__ int quot(int x) const {
    const int q = G == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), m));
    return q + (x - q * G >= G ? 1 : 0);
  }
};

// A tile that shares' borders cut, noted by the CTA that holds its first piece: the
// last CTA (-1: there is none), and which rows and heads they are.
struct PagedCut {
  int c1, row0, rho0, nG, head0;
};

struct PagedAttnParams {
  PagedView pv;
  int n_req, n_rows;
  Heads heads;
  const int32_t* row_off;
  const int32_t* pos0;
  const uint32_t* mask;
  int mask_ld;
  const __nv_bfloat16* q;
  long long q_ld;
  __nv_bfloat16* out;
  long long out_ld;
  float scale_log2;
  // a tile split between CTAs: two slots of partial rows per CTA (its first
  // tile and its last), unnormalised O and (max, sum) of each row, and arrival
  // counters per CTA for the tile that begins there and goes on
  float* part_o;                   // [grid][2][rows][hd]
  float2* part_ml;                 // [grid][2][rows]
  int* arrive;                     // [grid] (few rows)
  PagedCut* cut;                   // [grid] (many rows)
  int* status;
};

// Geometry of a kernel's work: TR query rows to a tile, KS keys to a step.  What a
// tile weighs when the work is shared out: TC for its beginning and end, and for
// each step 1, or 2 where the tile has more than HALF rows.  A share weighs MIN at
// least (little work leaves CTAs without any).  Measured, us:
//   256-row tiles, TC 4 / 8 / 12 / 16: 257 rows over 8192 slots 63 / 59 / 58 / 57, nine
//     ragged chunks at head size 64 49 / 45 / 44 / 46;
//   64-row tiles, TC 1 / 3 / 6 / 10: 32 requests of 16 rows 114 / 110 / 111 / 115;
//     MIN 1 / 3 / 5: 16 rows over 8192 slots 33 / 24 / 23, over 2048 17.6 / 17.1 / 19.3,
//     9 rows over 300 12.7 / 13.8 / 17.0;
//   16-row tiles, TC 2 .. 12: no difference; MIN 1 / 2 / 4: one row over 2048 slots 10.4 /
//     10.0 / 11.3, over 500 8.4 / 8.9 / 10.5, four rows over 2048 18.9 / 15.6 / -.
template <int TR_, int KS_, int TC_, int HALF_, int MIN_>
struct PagedGeo {
  static constexpr int TR = TR_, KS = KS_, TC = TC_, HALF = HALF_, MIN = MIN_;
  // Shares are whole multiples of the largest weight: every CTA between the first
  // and the last of a tile then holds a step of it.
  static constexpr int UNIT = HALF_ < TR_ ? 2 : 1;
};

// One request of the flattened work.  Its n rows and G heads of a KV head make
// n * G query rows (row = token * G + head), TR to a tile; tile j sees keys
// 0 .. key_end(j) - 1, in steps of KS keys.
struct PagedReq {
  int row0, n, p0, cap;
  bool masked;
  __device__ __forceinline__ void load(const PagedAttnParams& p, int r) {
    row0 = min(max(p.row_off[r], 0), p.n_rows);
    n = min(max(p.row_off[r + 1], row0), p.n_rows) - row0;
    cap = p.pv.table_ld << p.pv.page_shift;
    p0 = min(max(p.pos0[r], 0), cap);
    masked = p.mask != nullptr;
  }
  template <typename Geo>
  __device__ __forceinline__ int tiles(const Heads& h) const {
    return (n * h.G + Geo::TR - 1) / Geo::TR;
  }
  template <typename Geo>
  __device__ __forceinline__ int key_end(int j, const Heads& h) const {
    const int last = masked ? n - 1 : h.quot(min(j * Geo::TR + Geo::TR - 1, n * h.G - 1));
    return min(p0 + last + 1, cap);
  }
  template <typename Geo>
  __device__ __forceinline__ int weight(int j, const Heads& h) const {
    return min(n * h.G - j * Geo::TR, Geo::TR) > Geo::HALF ? 2 : 1;
  }
  // length of a tile, and of tiles [0, j1) of one KV head, on the line
  template <typename Geo>
  __device__ __forceinline__ int length(int j, const Heads& h) const {
    return Geo::TC + (key_end<Geo>(j, h) + Geo::KS - 1) / Geo::KS * weight<Geo>(j, h);
  }
  template <typename Geo>
  __device__ __forceinline__ long long lengths(int j1, const Heads& h) const {
    if (masked && j1 > 0) return (long long)(j1 - 1) * length<Geo>(0, h) + length<Geo>(j1 - 1, h);
    long long s = 0;
    for (int j = 0; j < j1; ++j) s += length<Geo>(j, h);
    return s;
  }
};

// A CTA's place on the line: requests, then KV heads, then query tiles, then, for
// each tile, TC units of overhead and its key steps.  The CTA's share is one
// stretch of the line; a step is its whose stretch holds the step's beginning.
struct PagedCursor {
  int r, g, j;             // request, KV head, tile
  int at, length, weight;  // place in the tile, its length, a step's weight
  long long left;          // what is left of the share
  int ctas;                // that have shares
  PagedReq rq;
};

// The key steps of the cursor's tile that lie in the share: [first, first + n) of
// `all`; they end `used` further on the line.
struct PagedPiece {
  int first, n, all, used;
  template <typename Geo>
  __device__ __forceinline__ static PagedPiece of(const PagedCursor& c) {
    PagedPiece p;
    p.used = static_cast<int>(min((long long)(c.length - c.at), c.left));
    auto steps = [&](int at) { return at <= Geo::TC ? 0 : (at - Geo::TC + c.weight - 1) / c.weight; };
    p.all = steps(c.length);
    p.first = steps(c.at);
    p.n = steps(c.at + p.used) - p.first;
    return p;
  }
};

// Whether some row of the cursor's tile sees one of the slots [t, end), where `end` is at
// most the end of what the tile's rows may see.  Warp-collective, and rare: asked only
// of slots that are not there.
template <typename Geo>
__device__ __forceinline__ bool paged_seen(const PagedAttnParams& p, const PagedCursor& c, int t, int end, int lane) {
  const PagedReq& rq = c.rq;
  if (t >= end) return false;
  if (!rq.masked || t < rq.p0) return true;                  // (causal: the last row sees them)
  const int b0 = t - rq.p0, b1 = static_cast<int>(min((long long)(end - rq.p0), 32ll * p.mask_ld));
  const int first = p.heads.quot(c.j * Geo::TR);
  const int last = p.heads.quot(min(c.j * Geo::TR + Geo::TR - 1, rq.n * p.heads.G - 1));
  bool sees = false;
  for (int i = first + lane; i <= last; i += 32) {
    const uint32_t* m = p.mask + (size_t)(rq.row0 + i) * p.mask_ld;
    for (int w = b0 >> 5; w * 32 < b1; ++w) {
      uint32_t u = m[w];
      if (w * 32 < b0) u &= 0xFFFFFFFFu << (b0 & 31);
      if (b1 - w * 32 < 32) u &= (1u << (b1 & 31)) - 1u;
      sees |= u != 0;
    }
  }
  return __any_sync(0xffffffffu, sees);
}

// An error if a row of the cursor's tile sees a slot past the table, or if the request
// begins before slot 0 or past the table.  Warp-collective.  (Nothing is kept for it from
// the plan on, and with tensor cores the issuing warp asks: a flag in PagedReq, or the
// question in the loading warp, made a prompt chunk take 249 us, not 239.)
template <typename Geo>
__device__ __forceinline__ void paged_past(const PagedAttnParams& p, const PagedCursor& c, int lane) {
  const PagedReq& rq = c.rq;
  if (rq.p0 > 0 && rq.p0 + rq.n <= rq.cap) return;
  const int rows = rq.masked ? rq.n : p.heads.quot(min(c.j * Geo::TR + Geo::TR - 1, rq.n * p.heads.G - 1)) + 1;
  if ((p.pos0[c.r] != rq.p0 || paged_seen<Geo>(p, c, rq.cap, rq.p0 + rows, lane)) && lane == 0)
    record_status(p.status, DFLASH_ERR_INVALID_ARG);
}

// a / b for a >= 0, b > 0; almost always within 32 bits, where it is quick.
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// Share of CTA c of `grid`: [paged_share(c), paged_share(c + 1)).
template <typename Geo>
__device__ __forceinline__ long long paged_share(long long total, int c, int grid) {
  const long long units = (total + Geo::UNIT - 1) / Geo::UNIT, q = div_pos(units, grid);
  return min((q * c + min((long long)c, units - q * grid)) * Geo::UNIT, total);
}
// The CTA whose share holds place s of the line.
template <typename Geo>
__device__ __forceinline__ int paged_owner(long long total, long long s, int grid) {
  const long long units = (total + Geo::UNIT - 1) / Geo::UNIT, q = div_pos(units, grid), m = units - q * grid;
  s /= Geo::UNIT;
  return static_cast<int>(s < m * (q + 1) ? div_pos(s, q + 1) : m + div_pos(s - m * (q + 1), q));
}

// Warp-collective: the line's length, the end of this CTA's share, and the place
// where the share begins.  Each lane adds up a run of requests; the run that holds
// the place is then searched by all lanes.
template <typename Geo>
__device__ __forceinline__ void paged_plan(const PagedAttnParams& p, int lane, long long* total_out,
                                           long long* end_out, PagedCursor* c) {
  const int run = (p.n_req + 31) / 32;
  auto length_of = [&](int r, PagedReq* q) {
    q->load(p, r);
    return q->lengths<Geo>(q->tiles<Geo>(p.heads), p.heads) * p.pv.n_kv;
  };
  auto scan = [&](long long v) {                           // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    return v;
  };
  PagedReq q = {};
  long long mine = 0;
  const int last = min((lane + 1) * run, p.n_req);
#pragma unroll 4
  for (int r = lane * run; r < last; ++r) mine += length_of(r, &q);
  long long upto = scan(mine);
  const long long total = __shfl_sync(0xffffffffu, upto, 31);
  c->ctas = static_cast<int>(min((long long)gridDim.x, max(div_pos(total, Geo::MIN), 1ll)));
  const long long begin = paged_share<Geo>(total, blockIdx.x, c->ctas);
  const long long end = paged_share<Geo>(total, blockIdx.x + 1, c->ctas);
  *total_out = total;
  *end_out = end;
  c->left = end - begin;
  if (c->left <= 0) return;
  // the lane whose run holds the place, and what lies before that run
  int l = __ffs(__ballot_sync(0xffffffffu, upto > begin)) - 1;
  long long before = __shfl_sync(0xffffffffu, upto - mine, l), length = __shfl_sync(0xffffffffu, mine, l);
  c->r = l;
  if (run == 1) {                                          // (q is the lane's own request)
    c->rq = q;
    c->rq.row0 = __shfl_sync(0xffffffffu, q.row0, l);
    c->rq.n = __shfl_sync(0xffffffffu, q.n, l);
    c->rq.p0 = __shfl_sync(0xffffffffu, q.p0, l);
    c->rq.cap = p.pv.table_ld << p.pv.page_shift;
    c->rq.masked = p.mask != nullptr;
  } else {
    const int stop = min((l + 1) * run, p.n_req);
    for (int r0 = l * run; r0 < stop; r0 += 32) {
      mine = r0 + lane < stop ? length_of(r0 + lane, &q) : 0;
      upto = scan(mine);
      const unsigned past = __ballot_sync(0xffffffffu, before + upto > begin);
      if (past) {
        l = __ffs(past) - 1;
        before += __shfl_sync(0xffffffffu, upto - mine, l);
        length = __shfl_sync(0xffffffffu, mine, l);
        c->r = r0 + l;
        break;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    c->rq.load(p, c->r);
  }
  const long long per_g = div_pos(length, p.pv.n_kv);
  long long rem = begin - before;
  c->g = static_cast<int>(div_pos(rem, per_g));
  rem -= (long long)c->g * per_g;
  int j = 0, len;
  while (true) {
    len = c->rq.length<Geo>(j, p.heads);
    if (rem < len) break;
    rem -= len;
    ++j;
  }
  c->j = j;
  c->at = static_cast<int>(rem);
  c->length = len;
  c->weight = c->rq.weight<Geo>(j, p.heads);
}

// Past the piece, to the next tile.
template <typename Geo>
__device__ __forceinline__ void paged_next(const PagedAttnParams& p, const PagedPiece& pc, PagedCursor* c) {
  c->left -= pc.used;
  if (c->left <= 0) return;
  if (++c->j >= c->rq.tiles<Geo>(p.heads)) {
    c->j = 0;
    if (++c->g >= p.pv.n_kv) {
      c->g = 0;
      do {
        if (++c->r >= p.n_req) return;
        c->rq.load(p, c->r);
      } while (c->rq.n == 0);
    }
  }
  c->at = 0;
  c->length = c->rq.length<Geo>(c->j, p.heads);
  c->weight = c->rq.weight<Geo>(c->j, p.heads);
}

// The CTAs that hold the steps of the cursor's tile, which begins at `tile0`.
template <typename Geo>
__device__ __forceinline__ void paged_owners(const PagedCursor& c, long long total, long long tile0, int all,
                                             int* c0, int* c1) {
  *c0 = paged_owner<Geo>(total, tile0 + Geo::TC, c.ctas);
  *c1 = paged_owner<Geo>(total, tile0 + Geo::TC + (long long)(all - 1) * c.weight, c.ctas);
}

// Bits of keys [b, b + 32) relative to the first new token: 1 = seen.
__device__ __forceinline__ uint32_t seen_word(const uint32_t* mrow, int mask_ld, int b) {
  if (b <= -32) return 0xFFFFFFFFu;                          // context
  const int w = b >> 5, sh = b & 31;                         // floor: w = -1 for b in (-32, 0)
  const uint32_t lo = w < 0 ? 0xFFFFFFFFu : (w < mask_ld ? __ldg(mrow + w) : 0u);
  const uint32_t hi = w + 1 < mask_ld ? __ldg(mrow + w + 1) : 0u;
  return __funnelshift_r(lo, hi, sh);
}
// The low n bits (n clamped to [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// Parts of a tile whose loads are in flight when they are joined (8 / 16 / 20: one row over
// 2048 slots 10.0 / 9.9 / 9.6 us, four rows 15.6 / 15.5 / 14.1, one over 500 9.0 / 9.2 / 9.3).
constexpr int kJoin = 20;

// SMs that the join of few rows has room for (the calls refuse more), and the bytes it takes.
constexpr int kMostSms = 160;
constexpr int paged_pairs(int rows, int per_sm) { return rows * static_cast<int>(sizeof(float2)) * per_sm * kMostSms; }

// The end of a piece of a tile of few rows: the states of its four warps, sO [4][ROWS][LD]
// unnormalised and sMl [4][ROWS] (max, sum), of which `live` rows count, become rows of
// out; or, where shares' borders cut the tile, a part of it, and the last of its CTAs to
// arrive joins the parts, in key order.  scratch: SCRATCH bytes, free once sO has been
// read: a pair for each row of as many parts as there may be CTAs, PER_SM to an SM (a long
// request's tile falls into a part for each).  Block-collective; sLast: one int.
template <int HD, int ROWS, int LD, int THREADS, int SCRATCH, int PER_SM, typename Geo>
__device__ __forceinline__ void paged_finish_small(const PagedAttnParams& p, const PagedCursor& c,
                                                   const PagedPiece& pc, long long total, long long end, int rho0,
                                                   int live, const float* sO, const float2* sMl, void* scratch,
                                                   int* sLast) {
  static_assert(SCRATCH >= paged_pairs(ROWS, PER_SM), "the join's scratch");
  const PagedReq& rq = c.rq;
  const int tid = threadIdx.x, head0 = c.g * p.heads.G;
  // a thread takes four columns of a row: HD / 4 neighbours make a row
  const int items = live * (HD / 4);
  auto write = [&](int row, int col, const float4& v, float L) {
    const int rho = rho0 + row, to = p.heads.quot(rho);
    const float inv = 1.f / L;                         // a row that saw no key: zeros
    *reinterpret_cast<uint2*>(p.out + (long long)(rq.row0 + to) * p.out_ld +
                              (long long)(head0 + rho - to * p.heads.G) * HD + col) =
        L == 0.f ? make_uint2(0, 0)
                 : make_uint2(mmas::pack_bf16(v.x * inv, v.y * inv), mmas::pack_bf16(v.z * inv, v.w * inv));
  };
  auto add = [](float4& a, float f, const float4& v) {
    a.x += f * v.x;
    a.y += f * v.y;
    a.z += f * v.z;
    a.w += f * v.w;
  };
  const bool whole = pc.n == pc.all;
  int c0 = 0, c1 = 0;
  if (!whole) paged_owners<Geo>(c, total, end - c.left - c.at, pc.all, &c0, &c1);
  const int bid = blockIdx.x;
  const size_t slot = (size_t)bid * 2 + (bid == c0 ? 1 : 0);
  for (int i = tid; i < items; i += THREADS) {
    const int row = i / (HD / 4), col = i % (HD / 4) * 4;
    float M = -CUDART_INF_F, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sMl[w * ROWS + row].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float2 ml = sMl[w * ROWS + row];
      if (ml.y == 0.f) continue;                       // this warp saw nothing for the row
      const float f = ex2(ml.x - M);
      L += f * ml.y;
      add(acc, f, *reinterpret_cast<const float4*>(sO + (w * ROWS + row) * LD + col));
    }
    if (whole) {
      write(row, col, acc, L);
    } else {
      *reinterpret_cast<float4*>(p.part_o + (slot * ROWS + row) * HD + col) = acc;
      if (col == 0) p.part_ml[slot * ROWS + row] = make_float2(M, L);
    }
  }
  if (!whole) {
    __threadfence();
    __syncthreads();
    if (tid == 0) *sLast = atomicAdd(p.arrive + c0, 1) == c1 - c0;
    __syncthreads();
    if (*sLast) {
      __threadfence();
      if (tid == 0) p.arrive[c0] = 0;                  // for the next call
      // the pieces' (max, sum) first, all at once, into the idle ring
      float2* sPart = reinterpret_cast<float2*>(scratch);
      const int parts = c1 - c0 + 1;
      for (int i = tid; i < parts * ROWS; i += THREADS) {
        const int cc = c0 + i / ROWS;
        sPart[i] = i % ROWS < live
                       ? __ldcg(p.part_ml + ((size_t)cc * 2 + (cc == c0)) * ROWS + i % ROWS)
                       : make_float2(-CUDART_INF_F, 0.f);
      }
      __syncthreads();
      for (int i = tid; i < items; i += THREADS) {
        const int row = i / (HD / 4), col = i % (HD / 4) * 4;
        float M = -CUDART_INF_F, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < parts; ++k) M = fmaxf(M, sPart[k * ROWS + row].x);
        for (int k0 = 0; k0 < parts; k0 += kJoin) {    // their loads in flight
          float4 v[kJoin];
#pragma unroll
          for (int k = 0; k < kJoin; ++k) {
            const int cc = c0 + min(k0 + k, parts - 1);
            v[k] = __ldcg(reinterpret_cast<const float4*>(
                p.part_o + (((size_t)cc * 2 + (cc == c0)) * ROWS + row) * HD + col));
          }
#pragma unroll
          for (int k = 0; k < kJoin; ++k) {
            const float2 ml = sPart[min(k0 + k, parts - 1) * ROWS + row];
            if (k0 + k >= parts || ml.y == 0.f) continue;
            const float f = ex2(ml.x - M);
            L += f * ml.y;
            add(acc, f, v[k]);
          }
        }
        write(row, col, acc, L);
      }
    }
  }
}

namespace {      // (a kernel of each file's own)

// Joins the tiles of NG groups of GT rows that shares' borders cut, each 32 rows (a lane to
// a row) to a block of eight warps, which share out the parts for the weights and the
// columns for the sums.
// Blocks x: the CTA that holds a tile's first piece.  (32 warps to a block, a warp for
// four columns, took longer: 128 rows over 4096 slots 32 us against 27.)
template <int HD, int NG, int GT>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedAttnParams p) {
  constexpr int kRound = 64, kFours = HD / 4, kCols = kFours / 8;
  constexpr int kAtOnce = 16 / kCols;                        // parts whose loads are in flight
  __shared__ float sF[kRound][32];
  __shared__ float sW[2][8][32];
  __shared__ __align__(16) uint2 sOut[32][kFours];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const PagedCut cut = p.cut[blockIdx.x];
  const int rho = cut.rho0 + blockIdx.y * 32 + lane;
  if (cut.c1 < 0 || rho - lane >= cut.nG) return;            // block-uniform
  const int c0 = blockIdx.x, parts = cut.c1 - c0 + 1;
  const int x = blockIdx.y * 32 / GT, row = blockIdx.y * 32 % GT + lane;
  const bool live = rho < cut.nG;
  auto at = [&](int k) { return ((size_t)(c0 + k) * 2 + (k == 0)) * NG + x; };
  auto ml_of = [&](int k) { return live ? __ldcg(p.part_ml + at(k) * GT + row) : make_float2(-CUDART_INF_F, 0.f); };
  float M = -CUDART_INF_F, L = 0.f;
  for (int k = warp; k < parts; k += 8) M = fmaxf(M, ml_of(k).x);
  sW[0][warp][lane] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) M = fmaxf(M, sW[0][w][lane]);
  float4 acc[kCols] = {};
  for (int r0 = 0; r0 < parts; r0 += kRound) {
    const int n = min(parts - r0, kRound);
    if (r0) __syncthreads();
    for (int k = warp; k < n; k += 8) {
      const float2 ml = ml_of(r0 + k);
      const float f = ml.y != 0.f ? ex2(ml.x - M) : -1.f;    // (-1: a part that saw no key)
      if (ml.y != 0.f) L += f * ml.y;
      sF[k][lane] = f;
    }
    __syncthreads();
    for (int k0 = 0; k0 < n; k0 += kAtOnce) {
      float4 v[kAtOnce][kCols];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                            (at(r0 + min(k0 + k, n - 1)) * kFours + warp * kCols) * GT + row;
#pragma unroll
        for (int j = 0; j < kCols; ++j) v[k][j] = __ldcg(src + j * GT);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float f = k0 + k < n ? sF[k0 + k][lane] : -1.f;
        if (f >= 0.f) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            acc[j].x += f * v[k][j].x;
            acc[j].y += f * v[k][j].y;
            acc[j].z += f * v[k][j].z;
            acc[j].w += f * v[k][j].w;
          }
        }
      }
    }
  }
  sW[1][warp][lane] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) L += sW[1][w][lane];
  const float inv = 1.f / L;
#pragma unroll
  for (int j = 0; j < kCols; ++j)                            // a row that saw no key: zeros
    sOut[lane][(warp * kCols + j) ^ (lane & 15)] =
        L == 0.f ? make_uint2(0, 0)
                 : make_uint2(mmas::pack_bf16(acc[j].x * inv, acc[j].y * inv),
                              mmas::pack_bf16(acc[j].z * inv, acc[j].w * inv));
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * kFours; i += 256) {
    const int r = i / kFours, ch = i % kFours, to = rho - lane + r;
    if (to >= cut.nG) break;
    const int tok = p.heads.quot(to), head = cut.head0 + to - tok * p.heads.G;
    reinterpret_cast<uint2*>(p.out + (long long)(cut.row0 + tok) * p.out_ld + (long long)head * HD)[ch] =
        sOut[r][ch ^ (r & 15)];
  }
}

}  // namespace

// Header, arrival counters, (max, sum) pairs, partial rows.
struct PagedWs {
  size_t arrive, cut, ml, o, bytes;
};
// Every kernel: kMostCtas CTAs an SM at most, one counter to a CTA (two where it has an SM
// alone), and for each SM two slots of 256 rows (or fewer rows to more CTAs).  One layout
// for all kernels and head sizes, so that calls which share a workspace find the counters
// where the others left zeros.
constexpr int kMostCtas = 3;
inline PagedWs paged_ws(int sms, int head_dim) {
  PagedWs w;
  const size_t rows = (size_t)sms * 2 * 256;
  w.arrive = 256;
  w.cut = w.arrive + align_up((size_t)sms * kMostCtas * sizeof(int), 256);
  w.ml = w.cut + align_up((size_t)sms * kMostCtas * sizeof(PagedCut), 256);
  w.o = w.ml + align_up(rows * sizeof(float2), 256);
  w.bytes = w.o + rows * head_dim * sizeof(float);
  return w;
}

}  // namespace dfl
