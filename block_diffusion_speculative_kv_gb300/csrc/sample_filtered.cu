// The target's token of every row from given random numbers, under temperature,
// top-k, top-p and min-p.
//
// "DFlash: Block Diffusion for Flash Speculative Decoding", section 3.4.4
// (verification at temperature 1) and "Accelerating Speculative Decoding with
// Block Diffusion Draft Trees", section 3.4.5 (the walk's target choices).
// With w_v = exp((l_v - max l) / T), the three filters keep a prefix of the
// tokens ordered by (logit desc, id asc), so the kept set is
//   { l_v > t }  and the first m tokens, by id, at l_v = t
// for one value t: top-k asks for the largest t with count(l >= t) >= k, top-p
// for the largest t whose mass(l >= t) reaches p of the mass that top-k kept,
// min-p gives t outright.  The draw is the first kept token, by id, whose
// cumulated mass passes u times the kept mass.
//
// One cluster of 2, 4 or 8 CTAs per row: each CTA keeps its slice of the row in
// shared memory (rows too long for that are read again from global memory), so HBM
// sees the logits once.  (Many long rows, whose slices would leave an SM one or two
// CTAs, are read again too.)  Counts and masses are whole numbers (a mass has 40
// fractional bits, every token's rounded for itself), so their sums over lanes, warps
// and CTAs do not depend on the order, every pass agrees with every other, and a row's
// result does not depend on the way it takes or on the size of its cluster.
//
// Two ways from there.  A small top-k (2 .. 512): the r-th best of a CTA's share of
// 2048 maxima over parts of the row, r = ceil(k / CTAs), is a value that r of its
// tokens reach, so k tokens of the row reach the least of the CTAs'; the few tokens
// that do are gathered in one CTA, ordered, and everything else happens on that list.
// Otherwise t is searched over the whole row by counting its tokens in bins
// (search() below), with one exponential per token for the whole mass and one for the
// mass above the border's surroundings.
//
// Neither bandwidth nor any unit bounds it, but the chain of block and cluster
// barriers between the steps of a row, of which an SM holds four CTAs: 480 rows of
// 151936 bf16 logits take 49 us greedy (6.3 waves of clusters; their bytes alone
// 21.5), 87 without filters, 92 with top-k 50, 251 with top-p 0.9 and 133 with
// filters of every kind mixed; one fp32 row takes 5 greedy, 12 with top-k 50, 13 with
// top-p and min-p on top of it and 33 with top-p 0.95 alone.
#include <math_constants.h>

#include "common.cuh"
#include "mma_sync.cuh"

namespace dfl {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxima = 8 * kThreads;              // parts of a row whose maxima are compared
constexpr int kMaxSlice = 196 * 1024;              // resident slice bytes
constexpr int kManySlice = 52 * 1024, kFewSlice = 40 * 1024;   // of three, four CTAs to an SM
constexpr int kListK = 512, kList = 1024;          // largest k, and tokens, of the gathered list
constexpr int kListPer = kList / kThreads;
constexpr int kBins = 1024;                        // of a search level (512: no faster, 256: 165 us, not 132)
constexpr int kNearRow = 8192;                     // tokens kept near the border, of a row
// A bin's weight bounds are widened by this much: exponents of up to 44 times a
// few roundings of 2^-24 stay below 2^-15.
constexpr float kSlack = 1e-4f;
constexpr float kOne = 1099511627776.f;            // 2^40
// More than the mass of all tokens that fit into near[].
constexpr uint64_t kTooMany = 1ull << 54;
static_assert(kNearRow < 1 << 14, "see above");

struct SampleParams {
  int vocab, part;          // part: elements of a warp's part, a multiple of 8
  long long ld;
  const void* logits;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t* tok;
  float* logp;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ uint32_t remote_addr(const void* p, uint32_t rank) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(ra)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return ra;
}
__device__ __forceinline__ uint64_t ld_remote(const uint64_t* p, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_remote(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote_addr(p, rank)) : "memory");
  return v;
}
// Sum and maximum over a warp: hardware reductions of 32-bit parts (22-bit ones for
// the sum, so that 32 of them do not overflow; the sum itself stays below 2^64).
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
  const uint32_t a = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) & 0x3FFFFFu);
  const uint32_t b = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 22) & 0x3FFFFFu);
  const uint32_t c = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 44));
  return a + ((uint64_t)b << 22) + ((uint64_t)c << 44);
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t h = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t l =
      __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32) == h ? static_cast<uint32_t>(v) : 0u);
  return ((uint64_t)h << 32) | l;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

struct Shared {
  uint64_t warp[2][kWarps];
  uint64_t xch[2][2];                    // exchanged between the CTAs, two in turn
  union {
    uint32_t hist[kBins];                // this CTA's counts
    uint64_t list[kList];                // gathered tokens: (ordered logit, ~id)
  };
  uint2 part[2][kWarps];
  uint32_t list_n;
  uint32_t found[2];
  uint64_t found_cum, before[2];
  uint64_t share[2];                     // measures of this CTA's share of the bins
  uint32_t near_n[kWarps];               // a warp's tokens near the border
  double below;                          // T ln(min-p), or 0: what min-p keeps reaches max + this
  float hi, lo;                          // log2(e) / T in two parts
};

// Sums (and maxima) over the cluster of CL CTAs; every thread receives the result.
// The exchange slots alternate, so one cluster barrier per reduction is enough.
template <int CL>
struct Reducer {
  Shared* s;
  int buf = 0;
  template <bool MAX>
  __device__ __forceinline__ void both(uint64_t& a, uint64_t& b) {
    auto op = [](uint64_t v) { return MAX ? warp_max(v) : warp_sum(v); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    a = op(a);
    b = op(b);
    if (lane == 0) {
      s->warp[0][warp] = a;
      s->warp[1][warp] = b;
    }
    __syncthreads();
    if (warp == 0) {
      const uint64_t x = op(lane < kWarps ? s->warp[0][lane] : 0);
      const uint64_t y = op(lane < kWarps ? s->warp[1][lane] : 0);
      if (lane == 0) {
        s->xch[buf][0] = x;
        s->xch[buf][1] = y;
      }
    }
    cluster_sync();
    a = op(lane < CL ? ld_remote(&s->xch[buf][0], lane) : 0);
    b = op(lane < CL ? ld_remote(&s->xch[buf][1], lane) : 0);
    buf ^= 1;
  }
};

// Weights of one row (mx finite): exp((x - mx) / T) as a power of two, log2(e) / T
// in two parts so that far tokens keep their relative precision; the second part
// is positive, so that an infinite distance never meets a zero or a sign.
struct Weight {
  float mx, hi, lo;
  __device__ __forceinline__ float operator()(float x) const {
    const float d = x - mx;
    return ex2(fmaf(d, hi, d * lo));
  }
  // two distances x - mx at once
  __device__ __forceinline__ float2 at(float2 d) const {
    const float2 y = __ffma2_rn(d, make_float2(hi, hi), __fmul2_rn(d, make_float2(lo, lo)));
    return make_float2(ex2(y.x), ex2(y.y));
  }
  __device__ __forceinline__ float2 dist(float a, float b) const {
    return __fadd2_rn(make_float2(a, b), make_float2(-mx, -mx));
  }
};
// Counts one at shared address a if lo <= x <= hi (no branch around it).
__device__ __forceinline__ void count_if_in(uint32_t a, float x, float lo, float hi) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ge.f32 p, %1, %2;\n\t"
      "setp.le.and.f32 p, %1, %3, p;\n\t"
      "@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(a),
      "f"(x), "f"(lo), "f"(hi)
      : "memory");
}
__device__ __forceinline__ void count_if_below(uint32_t a, float x, float limit) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.lt.f32 p, %1, %2;\n\t"
      "@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(a),
      "f"(x), "f"(limit)
      : "memory");
}
// A token's mass: its weight w in [0, 1] times 2^40, rounded, in two 32-bit conversions
// (64-bit ones are slow).
__device__ __forceinline__ uint64_t fix(float w) {
  const uint32_t h = __float2uint_rz(w * 1048576.f);                     // 2^20 steps
  const uint32_t l = __float2uint_rn(fmaf(-__uint2float_rn(h), 9.5367431640625e-7f, w) * kOne);
  return ((uint64_t)h << 20) + l;
}

// The sum of fix(w) over a thread's weights in [0, 1], a pair at a time and without a
// conversion: adding 12 (whose neighbours are 2^-20 apart) rounds w to 2^-20, adding
// 1.5 2^-17 (2^-40 apart) rounds what is left to 2^-40, and either sum's bits count the
// steps.  32 bits hold 2048 weights' steps, above or below; a thread has no more of a
// row of 2^22 tokens in a cluster of 8.
struct Masses {
  static constexpr float kHigh = 12.f, kLow = 1.1444091796875e-5f;   // kLow: 1.5 2^-17
  uint32_t high = 0, low = 0, n = 0;
  __device__ __forceinline__ void add(float2 w) {
    const float2 t = __fadd2_rn(w, make_float2(kHigh, kHigh));
    const float2 h = __fadd2_rn(t, make_float2(-kHigh, -kHigh));
    const float2 r = __fadd2_rn(__ffma2_rn(h, make_float2(-1.f, -1.f), w), make_float2(kLow, kLow));
    high += __float_as_uint(t.x) + __float_as_uint(t.y);
    low += __float_as_uint(r.x) + __float_as_uint(r.y);
    n += 2;
  }
  __device__ __forceinline__ uint64_t sum() const {
    const uint32_t h = high - n * __float_as_uint(kHigh);
    const int32_t l = static_cast<int32_t>(low - n * __float_as_uint(kLow));
    return ((uint64_t)h << 20) + static_cast<int64_t>(l);
  }
};

// The search runs over the ordered codes of the values (16 bits for bf16).
template <typename T>
struct Codes {
  static constexpr int kShift = sizeof(T) == 2 ? 16 : 0;
  static constexpr uint32_t kMinusZero = 0x7FFFFFFFu >> kShift;   // no token's: of() folds -0 onto +0
  __device__ static __forceinline__ uint32_t of(float x) { return ordered_bits(x) >> kShift; }
  __device__ static __forceinline__ float value(uint32_t c) {
    uint32_t k = c << kShift;
    if (kShift && !(k & 0x80000000u)) k |= 0xFFFFu;
    return from_ordered_bits(k);
  }
};

// Eight consecutive tokens as they lie in memory; a NaN never wins a maximum.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void gather(const __nv_bfloat16* p, int n) {   // n of them
    auto one = [&](int e) -> uint32_t { return e < n ? __bfloat16_as_ushort(p[e]) : 0xFF80u; };
    u = make_uint4(one(0) | one(1) << 16, one(2) | one(3) << 16, one(4) | one(5) << 16, one(6) | one(7) << 16);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void clean() {                // NaN becomes -inf
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
    const __nv_bfloat162 none = __float2bfloat162_rn(-CUDART_INF_F);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __hmax2(h[e], none);
  }
  __device__ __forceinline__ float max() const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void gather(const float* p, int n) {
    auto one = [&](int e) { return e < n ? p[e] : -CUDART_INF_F; };
    a = make_float4(one(0), one(1), one(2), one(3));
    b = make_float4(one(4), one(5), one(6), one(7));
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void clean() {
    float* h = &a.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = fmaxf(h[e], -CUDART_INF_F);
    h = &b.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = fmaxf(h[e], -CUDART_INF_F);
  }
  __device__ __forceinline__ float max() const {
    return fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

// A warp's part of the row, eight consecutive tokens to a lane and round.
template <typename T, bool RES>
struct Part {
  const T* data;        // shared memory (RES), or the row in global memory
  int id0, n;           // first token, tokens
  bool vec;             // 16-byte aligned
  __device__ __forceinline__ Chunk<T> at(int i) const {
    Chunk<T> c;
    if (RES || (vec && i + 8 <= n)) {
      c.load(data + i);
    } else {
      c.gather(data + i, n - i);
    }
    if constexpr (!RES) c.clean();
    return c;
  }
  __device__ __forceinline__ float one(int i) const {      // (not a NaN)
    return to_f32(data[i]);
  }
  // g(i, chunk) for every eight tokens; from global memory the next two rounds are
  // asked for ahead
  template <typename G>
  __device__ __forceinline__ void chunks(G g) const {
    int i = (threadIdx.x & 31) * 8;
    if constexpr (RES) {
#pragma unroll 2
      for (; i < n; i += 256) g(i, at(i));
    } else {
      Chunk<T> c[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) c[q] = at(min(i + q * 256, n));
      for (; i < n; i += 512) {
        Chunk<T> d[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) d[q] = at(min(i + (q + 2) * 256, n));
        g(i, c[0]);
        if (i + 256 < n) g(i + 256, c[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) c[q] = d[q];
      }
    }
  }
  // f(i, x) for every eight tokens (all), or for those of which one is at or above lo
  template <typename F>
  __device__ __forceinline__ void all(F f) const {
    chunks([&](int i, const Chunk<T>& c) {
      float x[8];
      c.get(x);
      f(i, x);
    });
  }
  template <typename F>
  __device__ __forceinline__ void each(float lo, F f) const {
    chunks([&](int i, const Chunk<T>& c) {
      if (!(c.max() >= lo)) return;
      float x[8];
      c.get(x);
      f(i, x);
    });
  }
};

// whole * f for f in [0, 1), rounded down; *rest: something was rounded away.
// (Whole numbers throughout: FP64 is slow on this GPU.)
__device__ __forceinline__ uint64_t share_of(uint64_t whole, float f, bool* rest) {
  *rest = false;
  if (!(f > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(f), e = bits >> 23;
  const uint64_t mant = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int sh = 150 - static_cast<int>(e ? e : 1);        // f = mant * 2^-sh, 24 <= sh <= 149
  const uint64_t lo = whole * mant, hi = __umul64hi(whole, mant);
  if (sh >= 64) {
    const int q = sh - 64;
    *rest = lo != 0 || (q < 64 && (hi & ((1ull << q) - 1))) || (q >= 64 && hi);
    return q < 64 ? hi >> q : 0;
  }
  *rest = (lo & ((1ull << sh) - 1)) != 0;
  return (hi << (64 - sh)) | (lo >> sh);
}
// u of the whole, as the last mass that the token must pass.
__device__ __forceinline__ uint64_t draw_target(float u, uint64_t whole) {
  if (u >= 1.f) return whole - 1;
  bool rest;
  return share_of(whole, u, &rest);
}
// The mass that top-p (p < 1) asks for.
__device__ __forceinline__ uint64_t mass_target(float p, uint64_t whole) {
  bool rest;
  const uint64_t t = share_of(whole, p, &rest);
  return max(t + (rest ? 1 : 0), static_cast<uint64_t>(1));
}
// ln of a token's share of the kept mass, which is m 2^e with m in [1, 2).
__device__ __forceinline__ float log_share(float x, float mx, float temp, uint64_t whole) {
  const int e = 63 - __clzll(whole);
  const float m = static_cast<float>(whole << (63 - e)) * 1.0842021724855044e-19f;   // 2^-63
  const float ln = fmaf(e - 40, 0.693145751953125f, fmaf(e - 40, 1.42860677e-6f, logf(m)));
  return (x == mx ? 0.f : (x - mx) / temp) - ln;
}

// Sum over the block of a mass of at most 2^40 per token, kListPer tokens a thread:
// two 20-bit halves, so that 32-bit sums hold 1024 tokens.  Calls alternate `turn`.
__device__ __forceinline__ uint64_t list_sum(uint32_t hi, uint32_t lo, Shared* s, int* turn) {
  const int warp = threadIdx.x >> 5;
  hi = __reduce_add_sync(0xffffffffu, hi);
  lo = __reduce_add_sync(0xffffffffu, lo);
  uint2* at = s->part[*turn];
  if ((threadIdx.x & 31) == 0) at[warp] = make_uint2(hi, lo);
  __syncthreads();
  uint32_t h = 0, l = 0;
#pragma unroll
  for (int x = 0; x < kWarps; ++x) {
    h += at[x].x;
    l += at[x].y;
  }
  *turn ^= 1;
  return ((uint64_t)h << 20) + l;
}

// Top-k, top-p, min-p and the draw on the n <= kThreads / 2 gathered tokens in
// s->list, of which k or more: a thread places its token among the others by
// counting the greater ones, and sums run in that order.  Block-collective.
__device__ __noinline__ void draw_sorted(const SampleParams& p, int row, Shared* s, int n, int k, float top_p,
                                         float min_p, float uf, float temp, const Weight& w) {
  const int tid = threadIdx.x;
  const uint64_t key = tid < n ? s->list[tid] : 0;
  const float x = from_ordered_bits(static_cast<uint32_t>(key >> 32));
  const uint32_t id = ~static_cast<uint32_t>(key);
  uint64_t* wt = s->list + kList / 2;
  const uint64_t mine = tid < n ? fix(w(x)) : 0;
  if (tid < n) wt[tid] = mine;
  __syncthreads();
  // the tokens before this one, and their mass; top-k keeps the first k
  int place = 0;
  uint64_t before = 0;
  if (tid < n) {
#pragma unroll 4
    for (int i = 0; i < n; ++i)
      if (s->list[i] > key) {
        ++place;
        before += wt[i];
      }
  }
  bool keep = tid < n && place < k;
  if (keep && place == k - 1) s->found_cum = before + mine;
  __syncthreads();
  const uint64_t target = top_p < 1.f ? mass_target(top_p, s->found_cum) : ~0ull;
  const float least = min_p > 0.f ? __double2float_ru(w.mx + s->below) : -CUDART_INF_F;
  keep = keep && (place == 0 || before < target) && x >= least;
  // cumulated by id, over what is kept
  wt[tid] = keep ? mine : 0;
  __syncthreads();
  if (tid >= n) return;
  uint64_t upto = 0, kept = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const uint64_t m = wt[i];
    kept += m;
    if (static_cast<uint32_t>(s->list[i]) >= static_cast<uint32_t>(key)) upto += m;   // ~id: ids up to this one
  }
  const uint64_t goal = draw_target(uf, kept);
  if (keep && upto - mine <= goal && goal < upto) {
    p.tok[row] = static_cast<int>(id);
    p.logp[row] = log_share(x, w.mx, temp, kept);
  }
}

// The same for a longer list in s->list; block-collective.  The border (t, m) as for a
// whole row, found by halving the range of codes; a thread holds kListPer tokens.
// (Counting costs n per token, halving some 50 block sums whatever n: 480 rows with
// top-k 50, about 70 tokens, 92 us counted and 113 halved, one fp32 row 12 and 18; 480 with
// top-k 400, about 450, 165 and 130.  The border between them is what half a block's
// threads hold.)
template <int SHIFT>
__device__ __noinline__ void draw_halving(const SampleParams& p, int row, Shared* s, int n, int k, float top_p,
                                         float min_p, float uf, float temp, float from, const Weight& w) {
  const int tid = threadIdx.x;
  uint32_t code[kListPer], id[kListPer];                   // (code 0: no token)
  uint64_t wt[kListPer];
  int turn = 0;
#pragma unroll
  for (int q = 0; q < kListPer; ++q) {
    const int i = q * kThreads + tid;
    const uint64_t key = i < n ? s->list[i] : 0;
    code[q] = static_cast<uint32_t>(key >> 32) >> SHIFT;
    id[q] = ~static_cast<uint32_t>(key);
    wt[q] = i < n ? fix(w(from_ordered_bits(static_cast<uint32_t>(key >> 32)))) : 0;
  }
  // what satisfies f: how many, or their mass
  auto count = [&](auto f) {
    uint32_t c = 0;
#pragma unroll
    for (int q = 0; q < kListPer; ++q) c += code[q] && f(q) ? 1 : 0;
    return static_cast<uint32_t>(list_sum(0, c, s, &turn));
  };
  auto mass = [&](auto f) {
    uint32_t h = 0, l = 0;
#pragma unroll
    for (int q = 0; q < kListPer; ++q)
      if (f(q)) {
        h += static_cast<uint32_t>(wt[q] >> 20);
        l += static_cast<uint32_t>(wt[q]) & 0xFFFFFu;
      }
    return list_sum(h, l, s, &turn);
  };
  const uint32_t top = ordered_bits(w.mx) >> SHIFT, floor = ordered_bits(from) >> SHIFT;
  uint32_t t = floor, hi = top;
  while (t < hi) {
    const uint32_t mid = t + (hi - t + 1) / 2;
    if (count([&](int q) { return code[q] >= mid; }) >= static_cast<uint32_t>(k)) t = mid;
    else hi = mid - 1;
  }
  uint32_t m = k - count([&](int q) { return code[q] > t; });
  if (top_p < 1.f) {
    const uint64_t above = mass([&](int q) { return code[q] > t; });
    const uint64_t one = fix(w(from_ordered_bits(t << SHIFT | (SHIFT && !(t >> 15) ? 0xFFFFu : 0u))));
    const uint64_t target = mass_target(top_p, above + m * one);
    if (target > above) {
      if (one) m = static_cast<uint32_t>(min(static_cast<uint64_t>(m), (target - above + one - 1) / one));
    } else {
      hi = top;
      while (t < hi) {
        const uint32_t mid = t + (hi - t + 1) / 2;
        if (mass([&](int q) { return code[q] >= mid; }) >= target) t = mid;
        else hi = mid - 1;
      }
      const uint64_t over = mass([&](int q) { return code[q] > t; });
      const uint64_t each = fix(w(from_ordered_bits(t << SHIFT | (SHIFT && !(t >> 15) ? 0xFFFFu : 0u))));
      m = each ? static_cast<uint32_t>((target - over + each - 1) / each) : 1;
    }
  }
  if (min_p > 0.f) {
    // (the least value that it keeps; between two codes it is the upper one's)
    const float least = __double2float_ru(w.mx + s->below);
    uint32_t c = ordered_bits(least) >> SHIFT;
    if (from_ordered_bits(c << SHIFT | (SHIFT && !(c >> 15) ? 0xFFFFu : 0u)) < least) ++c;
    if (c > t) {
      t = c - 1;
      m = 0;
    }
  }
  // the first m ties, by id
  uint32_t last = 0xFFFFFFFFu;
  if (m < count([&](int q) { return code[q] == t; })) {
    uint32_t lo = 0, up = p.vocab - 1;                     // the least id that m ties reach
    while (m && lo < up) {
      const uint32_t mid = lo + (up - lo) / 2;
      if (count([&](int q) { return code[q] == t && id[q] <= mid; }) >= m) up = mid;
      else lo = mid + 1;
    }
    last = lo;
  }
  bool keep[kListPer];
#pragma unroll
  for (int q = 0; q < kListPer; ++q)
    keep[q] = code[q] && (code[q] > t || (m && code[q] == t && id[q] <= last));
  // the draw: the least id whose cumulated mass passes the goal
  const uint64_t kept = mass([&](int q) { return keep[q]; });
  const uint64_t goal = draw_target(uf, kept);
  uint32_t lo = 0, up = p.vocab - 1;
  while (lo < up) {
    const uint32_t mid = lo + (up - lo) / 2;
    if (mass([&](int q) { return keep[q] && id[q] <= mid; }) > goal) up = mid;
    else lo = mid + 1;
  }
#pragma unroll
  for (int q = 0; q < kListPer; ++q)
    if (keep[q] && id[q] == lo) {
      p.tok[row] = static_cast<int>(lo);
      const float x = from_ordered_bits(code[q] << SHIFT | (SHIFT && !(code[q] >> 15) ? 0xFFFFu : 0u));
      p.logp[row] = log_share(x, w.mx, temp, kept);
    }
}

template <typename T, bool RES, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(kThreads, 4)
sample_filtered_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  using C = Codes<T>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kNear = kNearRow / (CL * kWarps);          // of a warp
  float* near = reinterpret_cast<float*>(smem) + warp * kNear;
  T* slice = reinterpret_cast<T*>(smem + kWarps * kNear * sizeof(float));
  const int rank = static_cast<int>(cluster_rank());
  const int row = blockIdx.x / CL;
  pdl_wait();
  pdl_trigger();

  const T* src = static_cast<const T*>(p.logits) + row * p.ld;
  const int part0 = min((rank * kWarps + warp) * (long long)p.part, (long long)p.vocab);
  Part<T, RES> part;
  part.id0 = part0;
  part.n = min(p.part, p.vocab - part0);
  part.vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
  part.data = src + part0;
  const float temp = p.temperature ? p.temperature[row] : 1.f;
  const int k = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  const float uf = p.u[row];

  // the slice into shared memory (all of a lane's copies in flight at once), where
  // each lane reads its own tokens only; and this thread's best value
  constexpr int kMine = kMaxima / (CL * kThreads);
  float mine[kMine];
  int where[kMine];                        // its first chunk
#pragma unroll
  for (int q = 0; q < kMine; ++q) mine[q] = -CUDART_INF_F, where[q] = 0;
  auto take = [&](int q, float v, int i) {
    where[q] = v > mine[q] ? i : where[q];
    mine[q] = fmaxf(mine[q], v);
  };
  if constexpr (RES) {
    const Part<T, false> g{part.data, part.id0, part.n, part.vec};
    T* own = slice + (size_t)warp * p.part;
    for (int i = lane * 8; i < part.n; i += 256) {
      if (part.vec && i + 8 <= part.n) {
        const uint32_t to = mmas::smem_u32(own + i);
        mmas::cp_async16(to, part.data + i, true);
        if constexpr (sizeof(T) == 4) mmas::cp_async16(to + 16, part.data + i + 4, true);
      } else {
        g.at(i).store(own + i);
      }
    }
    mmas::cp_async_commit();
    mmas::cp_async_wait<0>();
    part.data = own;
  }
  constexpr int kAhead = RES || kMine > 4 ? kMine : 4;     // rounds asked for at once
  for (int i = lane * 8; i < part.n; i += 256 * kAhead) {
    Chunk<T> c[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
      if (!RES || i + q * 256 < part.n) c[q] = part.at(min(i + q * 256, part.n));
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if constexpr (RES) {
        if (i + q * 256 >= part.n) continue;
        c[q].clean();
        c[q].store(const_cast<T*>(part.data) + i + q * 256);
      }
      take(q % kMine, c[q].max(), i + q * 256);
    }
  }
  if (tid == 0) {                          // (seen by all after the next block barrier)
    sh.list_n = 0;
    // log2(e) = 1.44269502 + 1.92596e-8: the quotient, rounded down, and its rest
    const float hi = __fdiv_rd(1.4426950216293335f, temp);
    sh.hi = fminf(fmaxf(hi, 1e-38f), 3e38f);               // (T = inf: all alike)
    sh.lo = hi > 3e38f ? 1e-38f : fmaxf((fmaf(-hi, temp, 1.4426950216293335f) + 1.925963033500e-8f) / temp, 1e-38f);
    if (temp > 0.f && min_p > 0.f)                         // (T = inf times ln 1 is no number)
      sh.below = min_p < 1.f ? static_cast<double>(temp) * log(static_cast<double>(min_p)) : 0.;
  }
  Reducer<CL> red{&sh};

  const bool greedy = !(temp > 0.f) || k == 1;
  // the row's best token, (value desc, id asc), and a value that k tokens reach
  uint64_t best = 0;
  {
    float top = mine[0];
#pragma unroll
    for (int q = 1; q < kMine; ++q) top = fmaxf(top, mine[q]);
    const float here = top;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (here == top && top > -CUDART_INF_F) {
      int id = 0x7FFFFFFF;
      if (greedy) {                                        // (nobody else asks which token it is)
        int i = part.n;
#pragma unroll
        for (int q = 0; q < kMine; ++q) i = mine[q] == top ? min(i, where[q]) : i;
        float x[8];
        part.at(i).get(x);
#pragma unroll
        for (int e = 7; e >= 0; --e)
          if (x[e] == top) id = part.id0 + i + e;
      }
      best = ((uint64_t)ordered_bits(top) << 32) | (uint32_t)~id;
    }
  }
  const bool listed = !greedy && k > 1 && k <= kListK && k < p.vocab;
  uint64_t reach_code = 0;
  if (listed) {
    const uint32_t r = (k + CL - 1) / CL;
    uint32_t code[kMine];                                  // (16 bits are enough)
#pragma unroll
    for (int q = 0; q < kMine; ++q) code[q] = ordered_bits(mine[q]) >> 16;
    uint32_t lo = 0, hi = ordered_bits(CUDART_INF_F) >> 16;
    int turn = 0;
    while (lo < hi) {                                      // block-uniform
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      uint32_t n;
      if constexpr (kMine == 1) {
        n = __syncthreads_count(code[0] >= mid);
      } else {
        uint32_t c = 0;
#pragma unroll
        for (int q = 0; q < kMine; ++q) c += code[q] >= mid ? 1 : 0;
        n = static_cast<uint32_t>(list_sum(0, c, &sh, &turn));
      }
      if (n >= r) lo = mid;
      else hi = mid - 1;
    }
    reach_code = 0xFFFFull - lo;                           // the least of the CTAs', as a maximum
  }
  red.template both<true>(best, reach_code);
  const float mx = best ? from_ordered_bits(static_cast<uint32_t>(best >> 32)) : -CUDART_INF_F;
  const int best_id = static_cast<int>(~static_cast<uint32_t>(best));
  if (mx == -CUDART_INF_F || greedy) {
    if (rank == 0 && tid == 0) {
      p.tok[row] = mx == -CUDART_INF_F ? -1 : best_id;
      p.logp[row] = mx == -CUDART_INF_F ? -CUDART_INF_F : 0.f;
    }
    cluster_sync();                        // nobody leaves while its slots are read
    return;
  }
  const Weight w{mx, sh.hi, sh.lo};

  if (listed && !isinf(mx)) {
    const float from = from_ordered_bits((0xFFFFu - static_cast<uint32_t>(reach_code)) << 16);
    if (from > -CUDART_INF_F) {
      part.each(from, [&](int i, const float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (x[e] >= from) {
            const uint32_t at = atomicAdd(&sh.list_n, 1u);
            if (at < kList)
              sh.list[at] = ((uint64_t)ordered_bits(x[e]) << 32) | (uint32_t) ~(part.id0 + i + e);
          }
      });
      __syncwarp();
      cluster_sync();
      uint32_t n = 0, n_mine = 0, n_before = 0;            // in all, of CTA `warp`, before it
#pragma unroll
      for (int r = 0; r < CL; ++r) {
        const uint32_t c = ld_remote(&sh.list_n, r);
        if (r < warp) n_before += c;
        if (r == warp) n_mine = c;
        n += c;
      }
      if (n <= kList) {
        static_assert(CL <= kWarps, "a warp takes a CTA's list");
        // (CTA 0's own tokens lie in front; the others' follow)
        if (rank == 0 && warp > 0)
          for (uint32_t i = lane; i < n_mine; i += 32) sh.list[n_before + i] = ld_remote(&sh.list[i], warp);
        __syncwarp();
        cluster_sync();                    // the lists are read: the other CTAs are done
        if (rank != 0) return;
        __syncthreads();
        if (n <= kThreads / 2) draw_sorted(p, row, &sh, static_cast<int>(n), k, top_p, min_p, uf, temp, w);
        else draw_halving<C::kShift>(p, row, &sh, static_cast<int>(n), k, top_p, min_p, uf, temp, from, w);
        return;
      }
      // more tokens than the list holds (long ties): search
      cluster_sync();                      // (the lists share their memory with the bins)
    }
  }

  // kept: x > t, and the first m tokens at x == t
  float t = -CUDART_INF_F;
  uint32_t m = 0;
  const uint32_t top_code = C::of(mx), floor_all = C::of(-CUDART_INF_F);

  // A search by mass leaves the mass of this thread's tokens above over_v, and (close)
  // the tokens between over_v and somewhat below the border in near[].
  uint64_t over_sum = 0;
  float over_v = CUDART_INF_F;
  bool close = false;
  struct Found {
    uint32_t code;
    uint64_t above, target;
  };
  // The largest code whose measure (count, or mass) over x >= its value reaches
  // the target, and the measure strictly above it.  The target is k, or, by mass,
  // top_p of the mass above `lo` (and `extra` more, which lies at lo; if that is
  // needed the answer is lo).  Each level counts the bracket's tokens in kBins
  // bins, first by distance from the best, up to `reach`, which spreads them
  // evenly, then by code.  By mass, a bin of the first level is taken at its middle's
  // weight; the bin that this points to and its neighbours make the next bracket,
  // whose tokens are few and are kept, and the masses above it and in it are then
  // summed exactly.  Should the border not lie there (or a warp's tokens not fit),
  // everything runs again with bounds: a bin's mass lies between its count times its
  // lightest and its heaviest weight, so a few bins remain.  Bins of one code settle it.
  auto search = [&](bool by_mass, uint32_t lo, uint64_t extra, float reach) {
    uint32_t hi = top_code;
    const uint32_t lo0 = lo;
    const float lo0_v = C::value(lo);
    uint64_t target = k;
    bool linear = reach < 1e30f, guess = by_mass && linear;
    close = false;
    if (by_mass && !linear) {              // the whole in a pass of its own
      Masses all;
      part.each(lo0_v, [&](int, const float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 y = w.at(w.dist(x[e], x[e + 1]));
          all.add(make_float2(x[e] > lo0_v ? y.x : 0.f, x[e + 1] > lo0_v ? y.y : 0.f));
        }
      });
      uint64_t whole = all.sum(), none = 0;
      red.template both<false>(whole, none);
      target = mass_target(top_p, whole + extra);
      if (target > whole) return Found{lo, whole, target};
    }
    while (true) {
      const float lo_v = C::value(lo), hi_v = C::value(hi);
      int shift = 0;
      while (((hi - lo) >> shift) >= kBins) ++shift;
      const float scale = static_cast<float>(kBins - 1) / reach;
      const float far_v = mx - reach;                      // (linear) beyond: the last bin
      for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
      if (lane == 0) sh.near_n[warp] = close ? sh.near_n[warp] : 0;
      __syncthreads();
      uint64_t sum = 0, in_sum = 0;
      Masses over;
      const uint32_t hist_c = mmas::smem_u32(sh.hist);
      // (no branch per token: nearly every warp has one in the bracket)
      auto bin_code = [&](float x) {
        count_if_in(hist_c + (((hi - C::of(x)) >> shift) << 2), x, lo_v, hi_v);
      };
      if (linear) {
        // the mass above lo, and the bins, in one pass; 2^23 + bin has the bin in its
        // low bits (rounded down)
        const uint32_t hist0 = hist_c - 0x4B000000u * 4u;  // 2^23 is 0x4B000000
        auto bin = [&](float d, bool in) {
          const float at = __fmaf_rd(d, -scale, 8388608.f);
          count_if_below(hist0 + __float_as_uint(at) * 4, in ? at : CUDART_INF_F, 8388608.f + (kBins - 1));
        };
        if (by_mass && lo0 == floor_all) {
          part.all([&](int, const float (&x)[8]) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 d = w.dist(x[e], x[e + 1]);
              over.add(w.at(d));
              bin(d.x, true);
              bin(d.y, true);
            }
          });
        } else {
          part.each(by_mass ? lo0_v : fmaxf(lo_v, far_v), [&](int, const float (&x)[8]) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 d = w.dist(x[e], x[e + 1]);
              if (by_mass) {
                const float2 y = w.at(d);
                over.add(make_float2(x[e] > lo0_v ? y.x : 0.f, x[e + 1] > lo0_v ? y.y : 0.f));
              }
              bin(d.x, x[e] >= lo_v);
              bin(d.y, x[e + 1] >= lo_v);
            }
          });
        }
        if (by_mass) sum = over.sum();
      } else if (close) {
        sum = over_sum;
        for (uint32_t i = lane; i < sh.near_n[warp]; i += 32) {
          const float x = near[i];
          if (x > hi_v) sum += fix(w(x));
          bin_code(x);
        }
      } else {
        part.each(lo_v, [&](int i, const float (&x)[8]) {
          if (by_mass) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 y = w.at(w.dist(x[e], x[e + 1]));
              over.add(make_float2(x[e] > hi_v ? y.x : 0.f, x[e + 1] > hi_v ? y.y : 0.f));
            }
          } else {
            uint32_t n8 = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) n8 += x[e] > hi_v ? 1 : 0;
            sum += n8;
          }
          if (guess) {
            uint32_t in = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (x[e] >= lo_v && x[e] <= hi_v) in |= 1u << e;
            for (; in; in &= in - 1) {
              const float y = part.one(i + __ffs(in) - 1);
              const uint32_t at = atomicAdd(&sh.near_n[warp], 1u);
              if (at < kNear) near[at] = y;
              in_sum += fix(w(y));
              bin_code(y);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) bin_code(x[e]);
          }
        });
        if (by_mass) {
          sum = over.sum();
          over_sum = sum;                                  // of this thread's tokens above hi_v
          over_v = hi_v;
        }
        __syncwarp();
        if (guess && lane == 0 && sh.near_n[warp] > kNear) in_sum += kTooMany;
      }
      __syncthreads();
      red.template both<false>(sum, in_sum);               // (all histograms are complete)
      if (linear && by_mass) {
        target = mass_target(top_p, sum + extra);
        if (target > sum) return Found{lo0, sum, target};
        sum = 0;                                           // nothing lies above the best
      }
      if (guess && !linear && !close) {
        close = sum < target && target <= sum + in_sum && in_sum < kTooMany;
        if (!close) {
          guess = false;
          linear = true;
          lo = lo0;
          hi = top_code;
          continue;
        }
      }
      const uint64_t above = sum;
      // Every CTA takes a share of the bins, from the best on; upper and lower bounds
      // (or the guess) of their measures
      constexpr int kShare = kBins / CL, kPer = kShare > kThreads ? kShare / kThreads : 1;
      const float per_bin = -w.hi / scale;                 // (linear) log2 of a bin's fall
      uint64_t up[kPer], low[kPer], cu = 0, cl = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        up[q] = low[q] = 0;
        if (kPer * tid + q >= kShare) continue;
        const uint32_t b = rank * kShare + kPer * tid + q;
        uint32_t n = 0;
#pragma unroll
        for (int r = 0; r < CL; ++r) n += ld_remote(&sh.hist[b], r);
        uint64_t wu = 1, wl = 1;
        if (linear && b == kBins - 1) {
          // what the bins did not count: at most everything
          n = p.vocab;
          wu = by_mass ? fix(ex2(-reach * w.hi) * (1.f + kSlack)) + 1 : 1;
          wl = 0;
        } else if (by_mass && n) {
          if (shift == 0 && !linear) {
            wu = wl = fix(w(C::value(hi - b)));
          } else if (linear && guess) {
            wu = fix(b ? ex2((b + 0.5f) * per_bin) : 1.f);   // (the best lies at its bin's edge)
          } else if (linear) {
            wu = fix(fminf(ex2(b * per_bin) * (1.f + kSlack), 1.f)) + 1;
            wl = fix(ex2((b + 1) * per_bin) * (1.f - kSlack));
          } else {
            const uint32_t top = hi - (b << shift), span = (1u << shift) - 1;
            wu = fix(fminf(w(C::value(top)) * (1.f + kSlack), 1.f)) + 1;
            wl = fix(w(C::value(top - lo > span ? top - span : lo)) * (1.f - kSlack));
          }
        }
        up[q] = n * wu;
        low[q] = n * wl;
        cu += up[q];
        cl += low[q];
      }
      const uint64_t wu_sum = warp_sum(cu), wl_sum = warp_sum(cl);
      if (lane == 0) {
        sh.warp[0][warp] = wu_sum;
        sh.warp[1][warp] = wl_sum;
      }
      __syncthreads();
      const uint64_t tu = lane < kWarps ? sh.warp[0][lane] : 0, tl = lane < kWarps ? sh.warp[1][lane] : 0;
      const uint64_t share_u = warp_sum(tu), share_l = warp_sum(tl);
      if (tid == 0) {
        sh.share[0] = share_u;
        sh.share[1] = share_l;
      }
      cluster_sync();
      // The first bin whose upper (lower) cumulated measure reaches the target (the
      // sums' roundings may leave it a little beyond everything): only the warp that
      // holds it looks closer.
      const uint64_t su = lane < CL ? ld_remote(&sh.share[0], lane) : 0;
      const uint64_t sl = lane < CL ? ld_remote(&sh.share[1], lane) : 0;
      const uint64_t goal = min(target, warp_sum(su) + above);
      const uint64_t end_u = warp_scan(su) + above, end_l = warp_scan(sl) + above;
      // the CTAs that hold them (none: 0, or everything)
      const unsigned in_u = __ballot_sync(0xffffffffu, lane < CL && end_u - su < goal && goal <= end_u);
      const unsigned in_l = __ballot_sync(0xffffffffu, lane < CL && end_l - sl < goal && goal <= end_l);
      const int cta_u = __ffs(in_u) - 1, cta_l = __ffs(in_l) - 1;
      if (cta_u == rank) {
        uint64_t at = __shfl_sync(0xffffffffu, end_u - su, cta_u) + warp_sum(lane < warp ? tu : 0);
        if (at < goal && goal <= at + wu_sum) {
          at += warp_scan(cu) - cu;
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            if (at < goal && goal <= at + up[q]) {
              sh.found[0] = rank * kShare + kPer * tid + q;
              sh.found_cum = at;
            }
            at += up[q];
          }
        }
      }
      if (cta_l == rank) {
        uint64_t at = __shfl_sync(0xffffffffu, end_l - sl, cta_l) + warp_sum(lane < warp ? tl : 0);
        if (at < goal && goal <= at + wl_sum) {
          at += warp_scan(cl) - cl;
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            if (at < goal && goal <= at + low[q]) sh.found[1] = rank * kShare + kPer * tid + q;
            at += low[q];
          }
        }
      }
      __syncwarp();
      cluster_sync();
      const uint32_t b1 = cta_u >= 0 ? ld_remote(&sh.found[0], cta_u) : 0;
      const uint32_t b2 = max(cta_l >= 0 ? ld_remote(&sh.found[1], cta_l) : kBins - 1, b1);
      const uint64_t cum = cta_u >= 0 ? ld_remote(&sh.found_cum, cta_u) : above;
      if (shift == 0 && !linear) return Found{hi - min(hi - lo, b1), cum, target};
      uint32_t nlo, nhi;
      if (linear) {
        // a little wider than the bins: the next level is exact about what lies above
        const float bin = 1.f / scale, more = guess ? 0.75f : 0.25f;
        const uint32_t last = guess ? b1 : b2;
        const float hv = __fsub_ru(mx, __fmul_rd(fmaxf(b1 - more, -1.f), bin));
        const float lv = __fsub_rd(mx, __fmul_ru(last + 1.f + more, bin));
        nhi = max(min(hi, C::of(hv)), lo);
        nlo = last + (guess ? 1 : 0) >= kBins - 1 ? lo : min(max(lo, C::of(lv)), nhi);
        linear = false;
      } else {
        nhi = hi - min(hi - lo, b1 << shift);
        nlo = hi - min(hi - lo, (b2 << shift) + ((1u << shift) - 1));
        if (nlo == lo && nhi == hi) {
          // no bin could be told from another: halve the bracket
          const uint32_t mid = lo + (hi - lo + 1) / 2;
          const float v = C::value(mid);
          uint64_t ge = 0, zero = 0;
          part.each(v, [&](int, const float (&x)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (x[e] >= v) ge += by_mass ? fix(w(x[e])) : 1;
          });
          red.template both<false>(ge, zero);
          if (ge >= target) nlo = mid;
          else nhi = mid - 1;
        }
      }
      // Tokens are told from the bracket by value, where -0 is 0, and counted by code: a
      // bracket that ended at the code of -0 would count the zeros in front of the bins.
      hi = nhi == C::kMinusZero ? nhi - 1 : nhi;
      lo = min(nlo, hi);
    }
  };

  if (isinf(mx)) {
    // the tokens at +inf share the mass: ties at the border, of which top-k takes
    // the first k and top-p their share
    uint64_t n = 0, none = 0;
    part.each(mx, [&](int, const float (&x)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) n += x[e] == mx ? 1 : 0;
    });
    __syncwarp();
    red.template both<false>(n, none);
    if (k > 1) n = min(n, static_cast<uint64_t>(k));
    if (top_p < 1.f) n = min(n, max(mass_target(top_p, n), static_cast<uint64_t>(1)));
    t = mx;
    m = static_cast<uint32_t>(n);
  } else {
    if (k > 1 && k < p.vocab) {
      const Found f = search(false, floor_all, 0, 32.f);
      t = C::value(f.code);
      if (t > -CUDART_INF_F) m = static_cast<uint32_t>(k - f.above);
    }
    if (top_p < 1.f) {
      Found f{top_code, 0, 0};
      const uint32_t floor_code = C::of(t);
      const uint64_t extra = m ? m * fix(w(t)) : 0;
      if (t < mx) {
        // tokens further than `reach` below the best weigh less than 1 - p together
        const float reach = fminf(mx - t, temp * logf(p.vocab / (1.f - fmaxf(top_p, 0.f))));
        f = search(true, floor_code, extra, fmaxf(reach, 1e-30f));
      } else {
        f.target = mass_target(top_p, extra);              // top-k left ties at the best alone
      }
      if (f.code > floor_code || m) {
        // how many of the ties at the border it takes
        const uint64_t one = fix(w(C::value(f.code)));
        uint64_t need = f.target > f.above && one ? (f.target - f.above + one - 1) / one : 1;
        if (f.code == floor_code && need > m) need = m;
        m = static_cast<uint32_t>(min(need, static_cast<uint64_t>(0xFFFFFFFFu)));
        t = C::value(f.code);
      }
    }
    if (min_p > 0.f) {
      const float least = __double2float_ru(mx + sh.below);
      if (least > t) {
        t = nextafterf(least, -CUDART_INF_F);
        m = 0;
      }
    }
  }
  // (the sum above over_v stands only if the border lies below it)
  if (t > over_v) over_v = CUDART_INF_F;
  if (over_v == CUDART_INF_F) {
    over_sum = 0;
    close = false;
  }

  // kept mass and ties of every part, in token order
  const uint64_t one = m ? (isinf(mx) ? fix(1.f) : fix(w(t))) : 0;
  uint64_t gt = over_sum;
  uint32_t ties = 0;
  if (t == -CUDART_INF_F) {
    Masses all;
    part.all([&](int, const float (&x)[8]) {               // nothing was filtered
#pragma unroll
      for (int e = 0; e < 8; e += 2) all.add(w.at(w.dist(x[e], x[e + 1])));
    });
    gt += all.sum();
  } else if (close) {
    for (uint32_t i = lane; i < sh.near_n[warp]; i += 32) {
      const float x = near[i];
      if (x > t) gt += fix(w(x));
      if (x == t) ++ties;
    }
  } else {
    Masses rest;
    part.each(t, [&](int, const float (&x)[8]) {
      uint32_t in = 0;                                     // above the border, not yet summed
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (x[e] > t && x[e] <= over_v) in |= 1u << e;
        if (x[e] == t) ++ties;
      }
      if (in) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 y = w.at(w.dist(x[e], x[e + 1]));
          rest.add(make_float2((in >> e) & 1u ? y.x : 0.f, (in >> e) & 2u ? y.y : 0.f));
        }
      }
    });
    gt += rest.sum();
  }
  __syncwarp();
  gt = warp_sum(gt);
  ties = __reduce_add_sync(0xffffffffu, ties);
  const int buf = red.buf;
  __syncthreads();
  if (lane == 0) {
    sh.warp[0][warp] = gt;
    sh.warp[1][warp] = ties;
  }
  __syncthreads();
  if (warp == 0) {
    const uint64_t x = warp_sum(lane < kWarps ? sh.warp[0][lane] : 0);
    const uint64_t y = warp_sum(lane < kWarps ? sh.warp[1][lane] : 0);
    if (lane == 0) {
      sh.xch[buf][0] = x;
      sh.xch[buf][1] = y;
    }
  }
  cluster_sync();
  uint64_t before_gt = 0, before_tie = 0, all_gt = 0, all_tie = 0;
#pragma unroll
  for (int r = 0; r < CL; ++r) {
    const uint64_t a = ld_remote(&sh.xch[buf][0], r), b = ld_remote(&sh.xch[buf][1], r);
    all_gt += a;
    all_tie += b;
    if (r < rank) {
      before_gt += a;
      before_tie += b;
    }
  }
  cluster_arrive();                        // nobody leaves while its slots are read
  for (int x = 0; x < warp; ++x) {
    before_gt += sh.warp[0][x];
    before_tie += sh.warp[1][x];
  }
  auto kept_ties = [&](uint64_t n) { return n < m ? n : static_cast<uint64_t>(m); };
  const uint64_t whole = all_gt + kept_ties(all_tie) * one;
  const uint64_t goal = draw_target(uf, whole);
  // The part whose cumulated mass passes the goal; all warps of its CTA look into it,
  // each into some rounds of 256 tokens.
  const uint64_t cum = before_gt + kept_ties(before_tie) * one;
  const uint64_t part_end = before_gt + gt + kept_ties(before_tie + ties) * one;
  if (tid == 0) sh.found[0] = kWarps;
  __syncthreads();
  if (lane == 0 && cum <= goal && goal < part_end) {
    sh.found[0] = warp;
    sh.before[0] = before_gt;
    sh.before[1] = before_tie;
  }
  __syncthreads();
  if (sh.found[0] < kWarps) {                              // block-uniform
    const int owner = sh.found[0];
    Part<T, RES> its = part;
    its.id0 = (rank * kWarps + owner) * p.part;            // (holds a token: below vocab)
    its.data = RES ? slice + (size_t)owner * p.part : src + its.id0;
    its.n = min(p.part, p.vocab - its.id0);
    const int rounds = (its.n + 255) / 256, r0 = rounds * warp / kWarps, r1 = rounds * (warp + 1) / kWarps;
    auto chunk = [&](int i, float (&x)[8], uint64_t& g, uint32_t& tie) {
      g = 0;
      tie = 0;
      if (i >= its.n) return;
      its.at(i).get(x);
      Masses above;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 y = w.at(w.dist(x[e], x[e + 1]));
        above.add(make_float2(x[e] > t ? y.x : 0.f, x[e + 1] > t ? y.y : 0.f));
        tie += (x[e] == t ? 1 : 0) + (x[e + 1] == t ? 1 : 0);
      }
      g = above.sum();
    };
    uint64_t sg = 0;
    uint32_t st = 0, tie;
    float x[8];
    for (int r = r0; r < r1; ++r) {
      uint64_t g;
      chunk(r * 256 + lane * 8, x, g, tie);
      sg += g;
      st += tie;
    }
    sg = warp_sum(sg);
    st = __reduce_add_sync(0xffffffffu, st);
    if (lane == 0) {
      sh.warp[0][warp] = sg;
      sh.warp[1][warp] = st;
    }
    __syncthreads();
    uint64_t cg = sh.before[0], ct = sh.before[1];         // before this warp's rounds
    for (int x = 0; x < warp; ++x) {
      cg += sh.warp[0][x];
      ct += sh.warp[1][x];
    }
    if (cg + kept_ties(ct) * one <= goal && goal < cg + sg + kept_ties(ct + st) * one) {
      for (int r = r0; r < r1; ++r) {                      // warp-uniform
        const int i = r * 256 + lane * 8;
        uint64_t g;
        chunk(i, x, g, tie);
        const uint64_t ig = warp_scan(g), it = warp_scan(tie);
        const bool past = cg + ig + kept_ties(ct + it) * one > goal;
        const unsigned any = __ballot_sync(0xffffffffu, past);
        if (any) {
          if (lane == __ffs(any) - 1) {
            const uint64_t t0 = ct + it - tie;
            uint64_t g0 = cg + ig - g;
            float got = 0.f;
            uint32_t seen = 0;
            int id = -1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const bool above = x[e] > t, at = x[e] == t;
              if (above) g0 += fix(w(x[e]));
              if (at) ++seen;
              if (id < 0 && (above || at) && g0 + kept_ties(t0 + seen) * one > goal) {
                id = its.id0 + i + e;
                got = x[e];
              }
            }
            p.tok[row] = id;
            p.logp[row] = log_share(got, mx, temp, whole);
          }
          break;
        }
        cg += __shfl_sync(0xffffffffu, ig, 31);
        ct += __shfl_sync(0xffffffffu, it, 31);
      }
    }
  }
  __syncwarp();
  cluster_wait();
}

template <typename T, bool RES, int CL>
void launch_cluster(SampleParams p, int rows, cudaStream_t st) {
  p.part = ((p.vocab + CL * kWarps - 1) / (CL * kWarps) + 7) / 8 * 8;
  const size_t near = kNearRow / CL * sizeof(float), slice = RES ? (size_t)kWarps * p.part * sizeof(T) : 0;
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (RES && (dev < 0 || dev >= 64 || !set[dev])) {
    cudaFuncSetAttribute(sample_filtered_kernel<T, RES, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         kMaxSlice + kWarps * 16 * sizeof(T) + near);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  launch_k(sample_filtered_kernel<T, RES, CL>, dim3(rows * CL), dim3(kThreads), near + slice, st, p);
}

template <typename T>
void launch_sample(const SampleParams& p, int rows, cudaStream_t st) {
  // Small clusters repeat less of a row's fixed work and leave room for more rows at
  // once, large ones are sooner done with a row: once there is a CTA to every SM, the
  // smallest cluster whose slices let several CTAs share an SM.  With top-p 0.9, bf16,
  // clusters of 8 / 4 / 2, us: 400 rows of 8192 122 / 57 / 38, of 50000 157 / 89 / 74, of
  // 100000 177 / 133 / 210, of 151936 213 / 202 / 282; 32 rows of 50000 23 / 22 / 27;
  // one row of 151936 25 / 31 / 48.  Slices of which few fit an SM are worse than none: 128
  // rows of 250000 118 resident in clusters of 8, 105 read again (from L2, mostly) in
  // clusters of 4; fp32, 400 rows of 151936 447 / 244.  At kFewSlice it depends on the
  // filters: bf16, 480 rows of 151936 (37 KB) with mixed filters 134 / 136, 400 with top-p
  // 0.9 213 / 188; fp32, 400 of 75000 with top-p 0.9 234 / 170.
  auto slice = [&](int cl) { return ((long long)p.vocab * (int)sizeof(T) + cl - 1) / cl; };
  auto fits = [&](int cl) { return (long long)rows * cl * 2 > num_sms() && slice(cl) <= kManySlice; };
  if (slice(8) > kMaxSlice)
    launch_cluster<T, false, 8>(p, rows, st);
  else if (!fits(4) && (slice(8) <= kFewSlice || (long long)rows * 4 <= num_sms()))
    launch_cluster<T, true, 8>(p, rows, st);
  else if (!fits(4))
    launch_cluster<T, false, 4>(p, rows, st);
  else if (!fits(2))
    launch_cluster<T, true, 4>(p, rows, st);
  else
    launch_cluster<T, true, 2>(p, rows, st);
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

dflash_status dflash_logits_sample_filtered(int rows, int vocab, long long ld, int dtype,
                                            const void* logits, const float* temperature,
                                            const int32_t* top_k, const float* top_p,
                                            const float* min_p, const float* u, int32_t* tok,
                                            float* logp, void* stream) {
  DFL_REQUIRE(rows >= 0 && rows <= (1 << 27), "sample filtered: need 0 <= rows <= 2^27");
  DFL_REQUIRE(vocab >= 1 && vocab <= (1 << 22) && ld >= vocab,
              "sample filtered: need 1 <= vocab <= min(ld, 2^22)");
  DFL_REQUIRE(dtype == DFLASH_F32 || dtype == DFLASH_BF16, "sample filtered: dtype must be F32 or BF16");
  if (rows == 0) return DFLASH_OK;
  DFL_REQUIRE(logits && u && tok && logp, "sample filtered: null logits/u/tok/logp");
  SampleParams p{};
  p.vocab = vocab;
  p.ld = ld;
  p.logits = logits;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.u = u;
  p.tok = tok;
  p.logp = logp;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope ts("sample_filtered", st);
    dtype == DFLASH_BF16 ? launch_sample<__nv_bfloat16>(p, rows, st) : launch_sample<float>(p, rows, st);
  }
  return check_launch("sample filtered");
}

}  // extern "C"
