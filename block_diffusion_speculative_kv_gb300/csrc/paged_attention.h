// Attention over a paged KV cache: parameters and work split shared by its
// kernels (paged_attention.cu).
#pragma once

#include "paged.cuh"

namespace dfl {

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

}  // namespace dfl
