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
#include <math_constants.h>

#include "common.cuh"

namespace dfl {

namespace {

constexpr int kCluster = 8, kThreads = 512, kWarps = kThreads / 32;
constexpr int kParts = kCluster * kWarps;          // contiguous parts of a row, one to a warp
constexpr int kMaxSlice = 200 * 1024;              // resident slice bytes
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
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint64_t ld_remote(const uint64_t* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), ra;
  uint64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(ra) : "memory");
  return v;
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

// Sums and maxima over the cluster; every thread receives the result.  The
// exchange slots alternate, so one cluster barrier per reduction is enough.
struct Shared {
  uint64_t warp[2][kWarps];
  uint64_t xch[2][2];
};
struct Reducer {
  Shared* s;
  int buf = 0;
  __device__ __forceinline__ void sum2(uint64_t& a, uint64_t& b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    a = warp_sum(a);
    b = warp_sum(b);
    if (lane == 0) {
      s->warp[0][warp] = a;
      s->warp[1][warp] = b;
    }
    __syncthreads();
    if (warp == 0) {
      const uint64_t x = warp_sum(lane < kWarps ? s->warp[0][lane] : 0);
      const uint64_t y = warp_sum(lane < kWarps ? s->warp[1][lane] : 0);
      if (lane == 0) {
        s->xch[buf][0] = x;
        s->xch[buf][1] = y;
      }
    }
    cluster_sync();
    a = warp_sum(lane < kCluster ? ld_remote(&s->xch[buf][0], lane) : 0);
    b = warp_sum(lane < kCluster ? ld_remote(&s->xch[buf][1], lane) : 0);
    buf ^= 1;
  }
  __device__ __forceinline__ uint64_t max1(uint64_t v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_max(v);
    if (lane == 0) s->warp[0][warp] = v;
    __syncthreads();
    if (warp == 0) {
      const uint64_t x = warp_max(lane < kWarps ? s->warp[0][lane] : 0);
      if (lane == 0) s->xch[buf][0] = x;
    }
    cluster_sync();
    v = warp_max(lane < kCluster ? ld_remote(&s->xch[buf][0], lane) : 0);
    buf ^= 1;
    return v;
  }
};

// Weights of one row: exp((x - mx) / T) as a power of two, log2(e) / T in two
// parts so that far tokens keep their relative precision.
struct Weight {
  float mx, hi, lo;
  __device__ __forceinline__ float operator()(float x) const {
    const float d = fmaxf(x - mx, -CUDART_MAX_NORMAL_F);   // finite: d * lo is then never NaN
    return x == mx ? 1.f : ex2(fmaf(d, hi, d * lo));
  }
};
__device__ __forceinline__ uint64_t fix(float w) { return __float2ull_rn(w * kOne); }

// Bisection runs over the ordered codes of the values (16 bits for bf16).
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

// A warp's part of the row, eight consecutive tokens to a lane and round.
template <typename T, bool RES>
struct Part {
  const T* data;        // shared memory (RES), or the row in global memory
  int id0, n;           // first token, tokens
  bool vec;             // 16-byte aligned
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31;
    for (int i = lane * 8; i < n; i += 256) {
      float x[8];
      get(i, x);
      f(i, x);
    }
  }
  __device__ __forceinline__ void get(int i, float (&x)[8]) const {
    if (RES || (vec && i + 8 <= n)) {
      if constexpr (sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(data + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = __uint_as_float(w[e] << 16);
          x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
      } else {
        const float4 a = reinterpret_cast<const float4*>(data + i)[0];
        const float4 b = reinterpret_cast<const float4*>(data + i)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = i + e < n ? to_f32<T>(data[i + e]) : -CUDART_INF_F;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaxf(x[e], -CUDART_INF_F);   // NaN counts as -inf
  }
};

template <typename T, bool RES>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
sample_filtered_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
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
  if constexpr (RES) {
    // the lane's own tokens: nobody else reads them before a barrier
    T* mine = reinterpret_cast<T*>(smem) + (size_t)warp * p.part;
    const T none = from_f32<T>(-CUDART_INF_F);
    for (int i = lane * 8; i < part.n; i += 256) {
      if (part.vec && i + 8 <= part.n) {
        const uint4* a = reinterpret_cast<const uint4*>(part.data + i);
        uint4* b = reinterpret_cast<uint4*>(mine + i);
#pragma unroll
        for (int e = 0; e < static_cast<int>(sizeof(T)) / 2; ++e) b[e] = __ldg(a + e);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[i + e] = i + e < part.n ? part.data[i + e] : none;
      }
    }
    part.data = mine;
  }
  Reducer red{&sh};

  // the best token: value desc, id asc
  uint64_t best = 0;
  part.each([&](int i, const float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint64_t k = ((uint64_t)ordered_bits(x[e]) << 32) | (uint32_t)~(part.id0 + i + e);
      if (i + e < part.n && k > best) best = k;
    }
  });
  best = red.max1(best);
  const float mx = from_ordered_bits(static_cast<uint32_t>(best >> 32));
  const int best_id = static_cast<int>(~static_cast<uint32_t>(best));
  const float temp = p.temperature ? p.temperature[row] : 1.f;
  const int k = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  if (mx == -CUDART_INF_F || !(temp > 0.f) || k == 1) {
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
  w.hi = isinf(mx) ? 1.f : static_cast<float>(c);   // +inf takes everything, at any T
  w.lo = isinf(mx) || isinf(w.hi) ? 0.f : static_cast<float>(c - static_cast<double>(w.hi));

  // kept: x > t, and the first m tokens at x == t
  float t = -CUDART_INF_F;
  uint32_t m = 0;
  const uint32_t top_code = Codes<T>::of(mx);
  auto count_ge = [&](float v) {
    uint64_t a = 0, b = 0;
    part.each([&](int, const float (&x)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a += x[e] >= v ? 1 : 0;
        b += x[e] > v ? 1 : 0;
      }
    });
    red.sum2(a, b);
    return make_ulonglong2(a, b);          // count(x >= v), count(x > v)
  };
  auto mass = [&](float v) {
    uint64_t a = 0, b = 0;
    part.each([&](int, const float (&x)[8]) {
      float ge = 0.f, gt = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = w(x[e]);
        ge += x[e] >= v ? y : 0.f;
        gt += x[e] > v ? y : 0.f;
      }
      a += fix(ge);
      b += fix(gt);
    });
    red.sum2(a, b);
    return make_ulonglong2(a, b);
  };

  if (k > 1 && k < p.vocab) {
    uint32_t lo = Codes<T>::of(-CUDART_INF_F), hi = top_code;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      if (count_ge(Codes<T>::value(mid)).x >= (uint64_t)k) lo = mid;
      else hi = mid - 1;
    }
    t = Codes<T>::value(lo);
    if (t > -CUDART_INF_F) m = static_cast<uint32_t>(k - count_ge(t).y);
  }
  if (top_p < 1.f) {
    const uint64_t gt = mass(t).y;
    const uint64_t whole = gt + (m ? m * fix(w(t)) : 0);
    const double want = static_cast<double>(top_p) * static_cast<double>(whole);
    const uint64_t target = want >= 1.0 ? static_cast<uint64_t>(ceil(want)) : 1;
    uint32_t lo = Codes<T>::of(t), hi = top_code;
    const uint32_t floor_code = lo;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      if (mass(Codes<T>::value(mid)).x >= target) lo = mid;
      else hi = mid - 1;
    }
    const bool moved = lo > floor_code;
    if (moved || m) {
      const float t2 = Codes<T>::value(lo);
      const uint64_t before = moved ? mass(t2).y : gt, one = fix(w(t2));
      uint64_t need = target > before && one ? (target - before + one - 1) / one : 1;
      if (!moved && need > m) need = m;
      m = static_cast<uint32_t>(need < 0xFFFFFFFFull ? need : 0xFFFFFFFFull);
      t = t2;
    }
  }
  if (min_p > 0.f) {
    const double v = static_cast<double>(mx) +
                     static_cast<double>(temp) * log(static_cast<double>(fminf(min_p, 1.f)));
    float f = static_cast<float>(v);       // the smallest fp32 value >= v
    if (static_cast<double>(f) < v) f = nextafterf(f, CUDART_INF_F);
    if (f > t) {
      t = nextafterf(f, -CUDART_INF_F);
      m = 0;
    }
  }

  // kept mass and ties of every part, in token order
  const uint64_t one = m ? fix(w(t)) : 0;
  uint64_t gt = 0;
  uint32_t ties = 0;
  auto chunk = [&](const float (&x)[8], uint32_t& tie) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s += x[e] > t ? w(x[e]) : 0.f;
      tie += x[e] == t ? 1 : 0;
    }
    return fix(s);
  };
  part.each([&](int, const float (&x)[8]) { gt += chunk(x, ties); });
  gt = warp_sum(gt);
  ties = __reduce_add_sync(0xffffffffu, ties);
  const int buf = red.buf;
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
  for (int r = 0; r < kCluster; ++r) {
    const uint64_t a = ld_remote(&sh.xch[buf][0], r), b = ld_remote(&sh.xch[buf][1], r);
    all_gt += a;
    all_tie += b;
    if (r < rank) {
      before_gt += a;
      before_tie += b;
    }
  }
  for (int x = 0; x < warp; ++x) {
    before_gt += sh.warp[0][x];
    before_tie += sh.warp[1][x];
  }
  auto kept_ties = [&](uint64_t n) { return n < m ? n : static_cast<uint64_t>(m); };
  const uint64_t whole = all_gt + kept_ties(all_tie) * one;
  const float uf = p.u[row];
  const double u = uf > 0.f ? (uf < 1.f ? static_cast<double>(uf) : 1.0) : 0.0;
  uint64_t target = static_cast<uint64_t>(u * static_cast<double>(whole));
  if (target >= whole) target = whole - 1;
  // the part whose cumulated mass passes the target
  uint64_t cum = before_gt + kept_ties(before_tie) * one;
  const uint64_t part_end = before_gt + gt + kept_ties(before_tie + ties) * one;
  if (cum <= target && target < part_end) {
    uint64_t cg = before_gt, ct = before_tie;          // before this round
    const int n = part.n;
    for (int i0 = 0; i0 < n; i0 += 256) {              // warp-uniform
      const int i = i0 + lane * 8;
      float x[8];
      uint32_t tie = 0;
      uint64_t g = 0;
      if (i < n) {
        part.get(i, x);
        g = chunk(x, tie);
      }
      uint64_t ig = g, it = tie;                       // inclusive scans
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t a = __shfl_up_sync(0xffffffffu, ig, o), b = __shfl_up_sync(0xffffffffu, it, o);
        if (lane >= o) {
          ig += a;
          it += b;
        }
      }
      const bool past = cg + ig + kept_ties(ct + it) * one > target;
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
            if (id < 0 && (above || at) && g0 + fix(s) + kept_ties(t0 + seen) * one > target) {
              id = part.id0 + i + e;
              got = x[e];
            }
          }
          p.tok[row] = id;
          // (x - max) / T - ln(kept mass)
          p.logp[row] = static_cast<float>(
              (got == mx ? 0.0 : (static_cast<double>(got) - static_cast<double>(mx)) / static_cast<double>(temp)) -
              log(static_cast<double>(whole) * (1.0 / 1099511627776.0)));
        }
        break;
      }
      cg += __shfl_sync(0xffffffffu, ig, 31);
      ct += __shfl_sync(0xffffffffu, it, 31);
    }
  }
  __syncwarp();
  cluster_sync();                          // nobody leaves while its slots are read
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
