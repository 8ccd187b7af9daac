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
// One cluster of 8 CTAs per row: each CTA keeps its slice of the row in shared
// memory (rows too long for that are read again from global memory), so HBM
// sees the logits once.  Counts and masses are whole numbers (a mass has 40
// fractional bits), so their sums over lanes, warps and CTAs do not depend on
// the order and every pass agrees with every other.
//
// Two ways from there.  A small top-k (2 .. 512): the r-th best of a CTA's
// per-thread maxima, r = ceil(k / 8), is a value that r of its tokens reach, so
// k tokens of the row reach the least of the eight; the few tokens that do are
// gathered in one CTA, sorted, and everything else happens on that list.
// Otherwise t is searched over the whole row by counting its tokens in bins
// (search() below).
#include <math_constants.h>

#include "common.cuh"

namespace dfl {

namespace {

constexpr int kCluster = 8, kThreads = 256, kWarps = kThreads / 32;
constexpr int kParts = kCluster * kWarps;          // contiguous parts of a row, one to a warp
constexpr int kMaxSlice = 200 * 1024;              // resident slice bytes
constexpr int kListK = 512, kList = 1024;          // largest k, and tokens, of the gathered list
constexpr int kBins = 1024;                        // of a search level
constexpr int kPer = kBins / kThreads;
// A bin's weight bounds are widened by this much: exponents of up to 44 times a
// few roundings of 2^-24 stay below 2^-15.
constexpr float kSlack = 1e-4f;
constexpr float kOne = 1099511627776.f;            // 2^40

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
__device__ __forceinline__ uint32_t add_remote(uint32_t* p, uint32_t rank, uint32_t n) {
  uint32_t v;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(v)
               : "r"(remote_addr(p, rank)), "r"(n)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_remote(uint64_t* p, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote_addr(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t t = __shfl_xor_sync(0xffffffffu, v, o);
    v = t > v ? t : v;
  }
  return v;
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
    struct {
      uint32_t hist[kBins];              // this CTA's counts
      uint32_t tot[kBins / kCluster];    // the cluster's, of this CTA's share of the bins
    };
    uint64_t list[kList];                // gathered tokens: (ordered logit, ~id)
  };
  uint32_t list_n;
  uint32_t found[2];
  uint64_t found_cum;
};

// Sums (and maxima) over the cluster; every thread receives the result.  The
// exchange slots alternate, so one cluster barrier per reduction is enough.
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
    a = op(lane < kCluster ? ld_remote(&s->xch[buf][0], lane) : 0);
    b = op(lane < kCluster ? ld_remote(&s->xch[buf][1], lane) : 0);
    buf ^= 1;
  }
};

// Weights of one row: exp((x - mx) / T) as a power of two, log2(e) / T in two
// non-negative parts so that far tokens keep their relative precision and no
// infinite distance meets a zero or a sign.  With mx = +inf, x - mx is NaN for
// the tokens there, and fminf turns that into 0.
struct Weight {
  float mx, hi, lo;
  __device__ __forceinline__ float operator()(float x) const {
    const float d = fminf(x - mx, 0.f);
    return ex2(fmaf(d, hi, d * lo));
  }
};
__device__ __forceinline__ uint64_t fix(float w) { return __float2ull_rn(w * kOne); }

// The search runs over the ordered codes of the values (16 bits for bf16).
template <typename T>
struct Codes {
  static constexpr int kShift = sizeof(T) == 2 ? 16 : 0;
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
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
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
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
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
      alignas(16) T t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = i + e < n ? data[i + e] : from_f32<T>(-CUDART_INF_F);
      c.load(t);
    }
    return c;
  }
  // f(i, x) for every eight tokens of which one is at or above lo (x: NaN counts as -inf)
  template <typename F>
  __device__ __forceinline__ void each(float lo, F f) const {
    for (int i = (threadIdx.x & 31) * 8; i < n; i += 256) {
      const Chunk<T> c = at(i);
      if (!(c.max() >= lo)) continue;
      float x[8];
      c.get(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaxf(x[e], -CUDART_INF_F);
      f(i, x);
    }
  }
};

// Bitonic sort of a[0 .. n), descending; n a power of two.  Block-collective.
__device__ __forceinline__ void sort_desc(uint64_t* a, int n) {
  for (int size = 2; size <= n; size <<= 1)
    for (int d = size >> 1; d; d >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < n / 2; i += kThreads) {
        const int x = 2 * i - (i & (d - 1)), y = x + d;
        const uint64_t p = a[x], q = a[y];
        if ((p < q) == ((x & size) == 0)) {
          a[x] = q;
          a[y] = p;
        }
      }
    }
  __syncthreads();
}
// Inclusive prefix sum of one value per thread and round, in thread order.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, Shared* s, uint64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_scan(v);
  __syncthreads();
  if (lane == 31) s->warp[0][warp] = v;
  __syncthreads();
  *total = 0;
  for (int x = 0; x < kWarps; ++x) {
    if (x < warp) v += s->warp[0][x];
    *total += s->warp[0][x];
  }
  return v;
}

// u of the whole, as the last mass that the token must pass.
__device__ __forceinline__ uint64_t draw_target(float uf, uint64_t whole) {
  const double u = uf > 0.f ? (uf < 1.f ? static_cast<double>(uf) : 1.0) : 0.0;
  const uint64_t t = static_cast<uint64_t>(u * static_cast<double>(whole));
  return t < whole ? t : whole - 1;
}
// ln of a token's share of the kept mass.
__device__ __forceinline__ float log_share(float x, float mx, float temp, uint64_t whole) {
  const double d = x == mx ? 0.0 : (static_cast<double>(x) - static_cast<double>(mx)) / static_cast<double>(temp);
  return static_cast<float>(d - log(static_cast<double>(whole) * (1.0 / 1099511627776.0)));
}
// The mass that top-p asks for.
__device__ __forceinline__ uint64_t mass_target(float p, uint64_t whole) {
  const double want = static_cast<double>(p) * static_cast<double>(whole);
  return want >= 1.0 ? static_cast<uint64_t>(ceil(want)) : 1;
}
// The least value that min-p keeps.
__device__ __forceinline__ float min_p_value(float min_p, float mx, float temp) {
  const double v = static_cast<double>(mx) + static_cast<double>(temp) * log(static_cast<double>(fminf(min_p, 1.f)));
  return __double2float_ru(v);
}

template <typename T, bool RES>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 4)
sample_filtered_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  using C = Codes<T>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank()), row = blockIdx.x / kCluster;
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

  // the slice into shared memory, where each lane reads its own tokens only
  float mine = -CUDART_INF_F;                              // this thread's best value
  {
    Part<T, false> g{part.data, part.id0, part.n, part.vec};
    T* own = reinterpret_cast<T*>(smem) + (size_t)warp * p.part;
#pragma unroll 4
    for (int i = lane * 8; i < part.n; i += 256) {
      const Chunk<T> c = g.at(i);
      if constexpr (RES) c.store(own + i);
      mine = fmaxf(mine, c.max());
    }
    if constexpr (RES) part.data = own;
  }
  if (tid == 0) sh.list_n = 0;
  Reducer red{&sh};

  // the row's best token, (value desc, id asc), and a value that k tokens reach
  uint64_t best = 0;
  {
    float top = mine;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (mine == top && top > -CUDART_INF_F) {
      int id = 0x7FFFFFFF;
      part.each(top, [&](int i, const float (&x)[8]) {
#pragma unroll
        for (int e = 7; e >= 0; --e)
          if (x[e] == top && part.id0 + i + e < id) id = part.id0 + i + e;
      });
      best = ((uint64_t)ordered_bits(top) << 32) | (uint32_t)~id;
    }
  }
  const bool greedy = !(temp > 0.f) || k == 1;
  const bool listed = !greedy && k > 1 && k <= kListK && k < p.vocab;
  uint64_t reach_code = 0;
  if (listed) {
    const int r = (k + kCluster - 1) / kCluster;
    const uint32_t code = C::of(mine);
    uint32_t lo = 0, hi = C::of(CUDART_INF_F);
    while (lo < hi) {                                      // block-uniform
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      if (__syncthreads_count(code >= mid) >= r) lo = mid;
      else hi = mid - 1;
    }
    reach_code = 0xFFFFFFFFull - lo;                       // the least of the eight, as a maximum
  }
  red.both<true>(best, reach_code);
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
  Weight w;
  w.mx = mx;
  const double c = 1.4426950408889634074 / static_cast<double>(temp);
  w.hi = isinf(mx) ? 1.f : fminf(__double2float_rd(c), 3e38f);   // +inf takes everything, at any T
  w.lo = isinf(mx) || c > 3e38 ? 1e-38f : fmaxf(static_cast<float>(c - static_cast<double>(w.hi)), 1e-38f);

  if (listed) {
    const float from = C::value(0xFFFFFFFFu - static_cast<uint32_t>(reach_code));
    if (from > -CUDART_INF_F) {
      part.each(from, [&](int i, const float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (x[e] >= from) {
            const uint32_t at = add_remote(&sh.list_n, 0, 1);
            if (at < kList)
              st_remote(&sh.list[at], 0,
                        ((uint64_t)ordered_bits(x[e]) << 32) | (uint32_t) ~(part.id0 + i + e));
          }
      });
      __syncwarp();
      cluster_sync();
      const int n = static_cast<int>(ld_remote(&sh.list_n, 0));
      if (n <= kList) {
        __syncwarp();
        cluster_arrive();
        if (rank != 0) return;             // (an exited CTA has arrived at every barrier)
        int size = 32;
        while (size < n) size <<= 1;
        for (int i = n + tid; i < size; i += kThreads) sh.list[i] = 0;
        sort_desc(sh.list, size);
        // weights in that order; what top-k keeps, then top-p and min-p
        const int rounds = (k + kThreads - 1) / kThreads;
        auto value = [&](int i) { return from_ordered_bits(static_cast<uint32_t>(sh.list[i] >> 32)); };
        uint64_t wt[kListK / kThreads] = {}, cum[kListK / kThreads] = {}, whole = 0;
#pragma unroll
        for (int q = 0; q < kListK / kThreads; ++q)
          if (q < rounds) {
            const int i = q * kThreads + tid;
            uint64_t all;
            wt[q] = i < k ? fix(w(value(i))) : 0;
            cum[q] = whole + block_scan(wt[q], &sh, &all);
            whole += all;
          }
        const uint64_t target = top_p < 1.f ? mass_target(top_p, whole) : ~0ull;
        const float least = min_p > 0.f ? min_p_value(min_p, mx, temp) : -CUDART_INF_F;
        // (the kept tokens are a prefix; the best is always among them)
        uint64_t kept = 0;
        uint32_t kept_n = 0;
#pragma unroll
        for (int q = 0; q < kListK / kThreads; ++q)
          if (q < rounds) {
            const int i = q * kThreads + tid;
            const bool keep = i < k && (i == 0 || cum[q] - wt[q] < target) && value(i) >= least;
            if (!keep) wt[q] = 0;
            kept_n += __syncthreads_count(keep);
            uint64_t all;
            block_scan(wt[q], &sh, &all);
            kept += all;
          }
        // by id: the weight travels as the place in the first order
        __syncthreads();
        uint64_t key[kListK / kThreads];
        int n2 = 32;
        while (n2 < static_cast<int>(kept_n)) n2 <<= 1;
#pragma unroll
        for (int q = 0; q < kListK / kThreads; ++q) {
          const int i = q * kThreads + tid;
          key[q] = i < static_cast<int>(kept_n) ? (sh.list[i] << 32) | (sh.list[i] >> 32) : 0;   // (~id, logit)
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kListK / kThreads; ++q)
          if (q * kThreads + tid < n2) sh.list[q * kThreads + tid] = key[q];
        sort_desc(sh.list, n2);
        const uint64_t goal = draw_target(uf, kept);
        uint64_t run = 0;
        for (int q = 0; q * kThreads < static_cast<int>(kept_n); ++q) {
          const int i = q * kThreads + tid;
          const float x = i < static_cast<int>(kept_n) ? from_ordered_bits(static_cast<uint32_t>(sh.list[i])) : 0.f;
          const uint64_t one = i < static_cast<int>(kept_n) ? fix(w(x)) : 0;
          uint64_t all;
          const uint64_t end = run + block_scan(one, &sh, &all);
          if (end - one <= goal && goal < end) {
            p.tok[row] = static_cast<int>(~static_cast<uint32_t>(sh.list[i] >> 32));
            p.logp[row] = log_share(x, mx, temp, kept);
          }
          run += all;
        }
        __syncwarp();
        cluster_wait();                    // the others have read list_n
        return;
      }
      // more tokens than the list holds (long ties): search
    }
  }

  // kept: x > t, and the first m tokens at x == t
  float t = -CUDART_INF_F;
  uint32_t m = 0;
  const uint32_t top_code = C::of(mx), floor_all = C::of(-CUDART_INF_F);

  struct Found {
    uint32_t code;
    uint64_t above, target;
  };
  // The largest code whose measure (count, or mass) over x >= its value reaches
  // the target, and the measure strictly above it.  The target is k, or, by mass,
  // top_p of the mass above `lo` (and `extra` more, which lies at lo; if that is
  // needed the answer is lo).  Each level counts the bracket's tokens in kBins
  // bins (first by distance from the best, up to `reach`, which spreads them
  // evenly; then by code) and takes the exact measure above the bracket.  A bin's
  // mass lies between its count times its lightest and its heaviest weight, so a
  // few bins, often one, remain.  Bins of one code settle it.
  auto search = [&](bool by_mass, uint32_t lo, uint64_t extra, float reach) {
    uint32_t hi = top_code;
    const uint32_t lo0 = lo;
    const float lo0_v = C::value(lo);
    uint64_t target = k;
    bool linear = !isinf(mx) && reach < 1e30f;
    if (by_mass && !linear) {              // the whole in a pass of its own
      uint64_t whole = 0, none = 0;
      part.each(lo0_v, [&](int, const float (&x)[8]) {
        float s8 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s8 += x[e] > lo0_v ? w(x[e]) : 0.f;
        whole += fix(s8);
      });
      red.both<false>(whole, none);
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
      __syncthreads();
      uint64_t sum = 0, none = 0;
      if (linear) {
        // the mass above lo, and the bins, in one pass
        part.each(by_mass ? lo0_v : fmaxf(lo_v, far_v), [&](int, const float (&x)[8]) {
          float s8 = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (by_mass) s8 += x[e] > lo0_v ? w(x[e]) : 0.f;
            const float at = (mx - x[e]) * scale;
            if (at < kBins - 1.f && x[e] >= lo_v) atomicAdd(&sh.hist[static_cast<uint32_t>(at)], 1u);
          }
          if (by_mass) sum += fix(s8);
        });
      } else {
        part.each(lo_v, [&](int, const float (&x)[8]) {
          float s8 = 0.f;
          uint32_t n8 = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (x[e] > hi_v) {
              if (by_mass) s8 += w(x[e]);
              else ++n8;
            } else if (x[e] >= lo_v) {
              atomicAdd(&sh.hist[(hi - C::of(x[e])) >> shift], 1u);
            }
          }
          sum += by_mass ? fix(s8) : n8;
        });
      }
      __syncthreads();
      red.both<false>(sum, none);                          // (all histograms are complete)
      if (linear && by_mass) {
        target = mass_target(top_p, sum + extra);
        if (target > sum) return Found{lo0, sum, target};
        sum = 0;                                           // nothing lies above the best
      }
      const uint64_t above = sum;
      if (tid < kBins / kCluster) {
        uint32_t n = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) n += ld_remote(&sh.hist[rank * (kBins / kCluster) + tid], r);
        sh.tot[tid] = n;
      }
      cluster_sync();
      // kPer bins to a thread, from the best on; upper and lower bounds of their measures
      uint64_t up[kPer], low[kPer], cu = 0, cl = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const uint32_t b = kPer * tid + q;
        uint32_t n = ld_remote(&sh.tot[b % (kBins / kCluster)], b / (kBins / kCluster));
        uint64_t wu = 1, wl = 1;
        if (linear && b == kBins - 1) {
          // what the bins did not count: at most everything
          n = p.vocab;
          wu = by_mass ? fix(ex2(-reach * w.hi) * (1.f + kSlack)) + 1 : 1;
          wl = 0;
        } else if (by_mass && n) {
          if (shift == 0 && !linear) {
            wu = wl = fix(w(C::value(hi - b)));
          } else if (linear) {
            wu = fix(fminf(ex2(-(b / scale) * w.hi) * (1.f + kSlack), 1.f)) + 1;
            wl = fix(ex2(-((b + 1) / scale) * w.hi) * (1.f - kSlack));
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
      uint64_t all, all_low;
      if (tid == 0) {
        sh.found[0] = 0;
        sh.found[1] = kBins - 1;
        sh.found_cum = above;
      }
      uint64_t at_u = block_scan(cu, &sh, &all) - cu + above;
      uint64_t at_l = block_scan(cl, &sh, &all_low) - cl + above;
      // the first bin whose upper (lower) cumulated measure reaches the target
      // (the sums' roundings may leave it a little beyond everything)
      const uint64_t goal = min(target, all + above);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (at_u < goal && goal <= at_u + up[q]) {
          sh.found[0] = kPer * tid + q;
          sh.found_cum = at_u;
        }
        if (at_l < goal && goal <= at_l + low[q]) sh.found[1] = kPer * tid + q;
        at_u += up[q];
        at_l += low[q];
      }
      __syncthreads();
      const uint32_t b1 = sh.found[0], b2 = max(sh.found[1], b1);
      const uint64_t cum = sh.found_cum;
      __syncthreads();
      if (shift == 0 && !linear) return Found{hi - min(hi - lo, b1), cum, target};
      uint32_t nlo, nhi;
      if (linear) {
        // a little wider than the bins: the next level is exact about what lies above
        const double bin = 1.0 / scale;
        const float hv = __double2float_ru(mx - (b1 - 0.125) * bin);
        const float lv = __double2float_rd(mx - (b2 + 1.125) * bin);
        nhi = max(min(hi, C::of(hv)), lo);
        nlo = b2 == kBins - 1 ? lo : min(max(lo, C::of(lv)), nhi);
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
            float s8 = 0.f;
            uint32_t n8 = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (x[e] >= v) {
                if (by_mass) s8 += w(x[e]);
                else ++n8;
              }
            ge += by_mass ? fix(s8) : n8;
          });
          red.both<false>(ge, zero);
          if (ge >= target) nlo = mid;
          else nhi = mid - 1;
        }
      }
      lo = nlo;
      hi = nhi;
    }
  };

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
      f.target = mass_target(top_p, extra);                // top-k left ties at the best alone
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
    const float least = min_p_value(min_p, mx, temp);
    if (least > t) {
      t = nextafterf(least, -CUDART_INF_F);
      m = 0;
    }
  }

  // kept mass and ties of every part, in token order
  const uint64_t one = m ? fix(w(t)) : 0;
  uint64_t gt = 0;
  uint32_t ties = 0;
  auto weigh = [&](const float (&x)[8], uint32_t& tie) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s += x[e] > t ? w(x[e]) : 0.f;
      tie += x[e] == t ? 1 : 0;
    }
    return fix(s);
  };
  part.each(t, [&](int, const float (&x)[8]) { gt += weigh(x, ties); });
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
  for (int r = 0; r < kCluster; ++r) {
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
  // the part whose cumulated mass passes the goal
  const uint64_t cum = before_gt + kept_ties(before_tie) * one;
  const uint64_t part_end = before_gt + gt + kept_ties(before_tie + ties) * one;
  if (cum <= goal && goal < part_end) {
    uint64_t cg = before_gt, ct = before_tie;          // before this round
    for (int i0 = 0; i0 < part.n; i0 += 256) {         // warp-uniform
      const int i = i0 + lane * 8;
      float x[8];
      uint32_t tie = 0;
      uint64_t g = 0;
      if (i < part.n) {
        part.at(i).get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaxf(x[e], -CUDART_INF_F);
        g = weigh(x, tie);
      }
      const uint64_t ig = warp_scan(g), it = warp_scan(tie);
      const bool past = cg + ig + kept_ties(ct + it) * one > goal;
      const unsigned any = __ballot_sync(0xffffffffu, past);
      if (any) {
        if (lane == __ffs(any) - 1) {
          const uint64_t g0 = cg + ig - g, t0 = ct + it - tie;
          float s = 0.f, got = 0.f;
          uint32_t seen = 0;
          int id = -1;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool above = x[e] > t, at = x[e] == t;
            if (above) s += w(x[e]);
            if (at) ++seen;
            if (id < 0 && (above || at) && g0 + fix(s) + kept_ties(t0 + seen) * one > goal) {
              id = part.id0 + i + e;
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
  __syncwarp();
  cluster_wait();
}

template <typename T>
void launch_sample(const SampleParams& p, int rows, cudaStream_t st) {
  const size_t slice = (size_t)kWarps * p.part * sizeof(T);
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(sample_filtered_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         kMaxSlice);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  if (slice <= kMaxSlice)
    launch_k(sample_filtered_kernel<T, true>, dim3(rows * kCluster), dim3(kThreads), slice, st, p);
  else
    launch_k(sample_filtered_kernel<T, false>, dim3(rows * kCluster), dim3(kThreads), 0, st, p);
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
  p.part = ((vocab + kParts - 1) / kParts + 7) / 8 * 8;
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
