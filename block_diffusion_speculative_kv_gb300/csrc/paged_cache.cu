// The rows that enter a paged KV cache: per-head RMSNorm and position rotation
// of queries and keys, and the append of keys and values into pages.
//
// norm_rope, per head x of hd elements at position p:
//   y = x / sqrt(mean(x^2) + eps) * gain,
//   out_i = y_i cos(p f_i) - y_{i+hd/2} sin(p f_i),
//   out_{i+hd/2} = y_{i+hd/2} cos(p f_i) + y_i sin(p f_i),  f_i = theta^(-2i/hd).
// Both operators read every element once and write it once: HBM bounds them
// (latency, for the rows of one decoding step).  A thread holds 8 elements of
// the first half of a head and their partners of the second, two 16-byte loads
// (bf16), so hd / 16 lanes share a head and the sum of squares is a shuffle
// over them.  It asks for all its heads of a batch of rows before it works on
// the first: one head at a time left HBM half idle.  A batch's cosines and sines
// are formed once by the CTA, while the loads are in flight.  Angles are whole
// numbers: a frequency is kept as turns per position, a 64-bit fraction, so p f_i
// modulo a turn is one 64-bit product whose overflow is the reduction (off by
// p 2^-64 turns and the frequency's 53 bits).
#include <cmath>

#include <cuda_fp8.h>
#include <math_constants.h>

#include "kernels.h"
#include "paged.cuh"

namespace dfl {

dflash_status check_pages(const dflash_pages* p, int n_req, const char* what, PagedView* out) {
  DFL_REQUIRE(p, "%s: null pages", what);
  DFL_REQUIRE(p->dtype == DFLASH_F32 || p->dtype == DFLASH_BF16, "%s: dtype must be F32 or BF16",
              what);
  DFL_REQUIRE(p->head_dim == 64 || p->head_dim == 128, "%s: head_dim must be 64 or 128", what);
  DFL_REQUIRE(p->page_size >= 16 && p->page_size <= 1024 &&
                  (p->page_size & (p->page_size - 1)) == 0,
              "%s: page_size must be a power of two in [16, 1024]", what);
  DFL_REQUIRE(p->n_kv >= 1 && p->n_pages >= 1 && p->table_ld >= 1,
              "%s: need n_kv, n_pages and table_ld >= 1", what);
  DFL_REQUIRE((long long)p->table_ld * p->page_size <= (1ll << 30),
              "%s: a request's slots exceed 2^30", what);      // (and rows added do not pass 2^31)
  DFL_REQUIRE((long long)p->n_pages * p->n_kv * p->page_size < (1ll << 31),
              "%s: the pool's rows exceed 2^31", what);
  DFL_REQUIRE(p->k && p->v && (p->table || n_req == 0), "%s: null pool or table", what);
  DFL_REQUIRE(((reinterpret_cast<uintptr_t>(p->k) | reinterpret_cast<uintptr_t>(p->v)) & 15) == 0,
              "%s: pools must be 16-byte aligned", what);
  *out = PagedView{p->k, p->v, p->table, p->table_ld, p->n_pages, log2_int(p->page_size), p->n_kv};
  return DFLASH_OK;
}

dflash_status check_pages(const dflash_pages_e4m3* p, int n_req, const char* what, PagedView* out) {
  DFL_REQUIRE(p, "%s: null pages", what);
  const dflash_pages same = {p->k,         p->v,    p->table,    p->table_ld, p->n_pages,
                             p->page_size, p->n_kv, p->head_dim, DFLASH_BF16};
  const dflash_status s = check_pages(&same, n_req, what, out);
  if (s) return s;
  DFL_REQUIRE(p->k_scale && p->v_scale, "%s: null scales", what);
  return DFLASH_OK;
}

namespace {

// Rotary frequencies theta^(-2i/head_dim) in turns, times 2^64.
struct RopeTurns {
  uint64_t f[64];
};
// (kept from call to call: 64 powers cost the host as much as the launch)
const RopeTurns& rope_turns(float theta, int head_dim) {
  static thread_local struct {
    float theta = 0.f;
    int head_dim = 0;
    RopeTurns t;
  } last;
  if (last.theta == theta && last.head_dim == head_dim) return last.t;
  const RopeFreqs fr = rope_freqs(theta, head_dim);
  RopeTurns& t = last.t;
  last.theta = theta;
  last.head_dim = head_dim;
  for (int i = 0; i < head_dim / 2; ++i) {
    const double turns = fr.f[i] / 6.283185307179586476925;
    t.f[i] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));   // whole turns are none
  }
  return t;
}
// (cos, sin) at a position >= 0.
__device__ __forceinline__ float2 turn_cs(int pos, uint64_t f) {
  const uint64_t a = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * f;
  // signed half turns in [-1, 1)
  const float x = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077392578125e-10f;   // 2^-31
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c, s);
}

// Eight consecutive elements as they lie in memory.  VEC: 16-byte aligned.
template <typename T>
struct Eight {
  uint4 u[sizeof(T) / 2];
  template <bool VEC>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];   // (in place: not __ldg)
    } else {
      T* t = reinterpret_cast<T*>(u);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = p[i];
    }
  }
  template <bool VEC>
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
    } else {
      const T* t = reinterpret_cast<const T*>(u);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = t[i];
    }
  }
  // as four pairs, for the packed fp32 instructions
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    } else {
      const float2* t = reinterpret_cast<const float2*>(u);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = t[i];
    }
  }
  __device__ __forceinline__ void set(const float2 (&x)[4]) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      u[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float2* t = reinterpret_cast<float2*>(u);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = x[i];
    }
  }
};

// The cosines and sines of a row, laid out so that the lanes of a head read 16-byte
// pieces (two cosines, two sines) next to one another: entry i belongs to lane i / 8.
template <int HD>
struct Turns {
  float4 v[4][HD / 16];
  __device__ __forceinline__ void put(int i, float2 c) {
    float* p = reinterpret_cast<float*>(&v[(i & 7) >> 1][i >> 3]) + (i & 1);
    p[0] = c.x;
    p[2] = c.y;
  }
  __device__ __forceinline__ void rotate(float2 (&a)[4], float2 (&b)[4], int sub) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 c = v[j][sub];
      const float2 cc = make_float2(c.x, c.y), ss = make_float2(c.z, c.w), ms = make_float2(-c.z, -c.w);
      const float2 x = a[j];
      a[j] = __ffma2_rn(x, cc, __fmul2_rn(b[j], ms));
      b[j] = __ffma2_rn(b[j], cc, __fmul2_rn(x, ss));
    }
  }
};

// i / n for 0 <= i < 2^31 / n, with m = divide_by(n).  A CTA divides i < 8 n (its
// rows' heads), so n may be 2^14 (kMaxHeads, below).
struct DivideBy {
  uint32_t n, m;
  __device__ __forceinline__ int operator()(int i) const {
    return n == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), m));
  }
};
DivideBy divide_by(int n) {
  return DivideBy{static_cast<uint32_t>(n), static_cast<uint32_t>(((1ull << 32) + n - 1) / n)};
}

constexpr int kThreads = 256;
// Rows of a CTA: several where there are enough of them to fill the SMs, one
// otherwise, for latency.  Measured with 32 + 8 heads of 128, bf16: norm and rotation
// of 512 rows 5.0 us one to a CTA and 7.2 us eight to a CTA, of 1024 rows 8.2 and
// 7.2, of 8197 rows 58.7 and 30.0 (5.6 TB/s); the append of 8 heads 3.2 and 3.8, 4.7
// and 4.0, 24.8 and 14.9.
constexpr int kNormRows = 8, kAppendRows = 8;
constexpr int kMaxHeads = 1 << 14;
static_assert((long long)kNormRows * kMaxHeads * kMaxHeads <= 1ll << 31 && kAppendRows <= kNormRows, "DivideBy");

struct NormRopeParams {
  int n_rows, n_q, n_kv;
  DivideBy by_q, by_kv;
  const void *q_gain, *k_gain;
  float eps;
  int rotate;
  RopeTurns fr;
  const int32_t* pos;
  const void *q, *k;
  void *q_out, *k_out;
  long long q_ld, k_ld, q_out_ld, k_out_ld;
};

// ROWS rows to a CTA, queries then keys; an item is a row's head, HD / 16 lanes to it
// (a warp's shuffle groups never straddle items, and lanes without one take part in
// the shuffles).
template <typename T, int HD, bool VEC, int ROWS>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope_kernel(const NormRopeParams p) {
  constexpr int kLanes = HD / 16, kHalf = HD / 2, kItems = kThreads / kLanes;
  constexpr int kBatch = 2;
  __shared__ Turns<HD> cs[ROWS];
  __shared__ int pos[ROWS];
  const int row0 = blockIdx.x * ROWS, tid = threadIdx.x, sub = tid % kLanes;
  const int rows = min(ROWS, p.n_rows - row0);
  pdl_wait();
  pdl_trigger();
  bool turned = false;
  auto part = [&](int heads, DivideBy by_heads, const void* in, long long ld, void* out, long long out_ld,
                  const void* gain) {
    const int items = rows * heads;
    if (items == 0) return;                                // block-uniform
    Eight<T> g[2] = {};
    if (gain) {
      g[0].template load<VEC>(static_cast<const T*>(gain) + 8 * sub);
      g[1].template load<VEC>(static_cast<const T*>(gain) + kHalf + 8 * sub);
    }
    for (int i0 = 0; i0 < items; i0 += kBatch * kItems) {  // block-uniform
      Eight<T> a[kBatch], b[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kItems + tid / kLanes, r = by_heads(i);
        if (i >= items) continue;
        const T* src = static_cast<const T*>(in) + (row0 + r) * ld + (i - r * heads) * HD + 8 * sub;
        a[k].template load<VEC>(src);
        b[k].template load<VEC>(src + kHalf);
      }
      if (!turned) {
        turned = true;
        for (int i = tid; i < ROWS * kHalf; i += kThreads) {
          const int r = i / kHalf, at = r < rows && p.pos ? p.pos[row0 + r] : 0;
          if (i % kHalf == 0) pos[r] = at;
          if (p.rotate) cs[r].put(i % kHalf, turn_cs(at, p.fr.f[i % kHalf]));
        }
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kItems + tid / kLanes, r = by_heads(i);
        const bool live = i < items && pos[r] >= 0;
        float2 x[4] = {}, y[4] = {};
        if (live) {
          a[k].get(x);
          b[k].get(y);
        }
        if (gain) {                                        // block-uniform
          float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(x[j], x[j], __ffma2_rn(y[j], y[j], s2));
          float ss = s2.x + s2.y;
#pragma unroll
          for (int off = kLanes / 2; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          const float inv = rsqrtf(ss * (1.f / HD) + p.eps);
          const float2 inv2 = make_float2(inv, inv);
          float2 gx[4], gy[4];
          g[0].get(gx);
          g[1].get(gy);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] = __fmul2_rn(__fmul2_rn(x[j], inv2), gx[j]);
            y[j] = __fmul2_rn(__fmul2_rn(y[j], inv2), gy[j]);
          }
        }
        if (!live) continue;
        if (p.rotate) cs[r].rotate(x, y, sub);
        a[k].set(x);
        b[k].set(y);
        T* dst = static_cast<T*>(out) + (row0 + r) * out_ld + (i - r * heads) * HD + 8 * sub;
        a[k].template store<VEC>(dst);
        b[k].template store<VEC>(dst + kHalf);
      }
    }
  };
  // (a single row's queries and keys go to two CTAs, at once)
  if (ROWS > 1 || blockIdx.y == 0) part(p.n_q, p.by_q, p.q, p.q_ld, p.q_out, p.q_out_ld, p.q_gain);
  if (ROWS > 1 || blockIdx.y == 1) part(p.n_kv, p.by_kv, p.k, p.k_ld, p.k_out, p.k_out_ld, p.k_gain);
}

struct AppendParams {
  PagedView pv;
  int n_req, n_rows;
  DivideBy by_heads;
  const int32_t *row_off, *pos0, *pos;
  const void *k, *v;
  long long kv_ld;
  int rotate;
  RopeTurns fr;
};

// ROWS rows to a CTA, whose places in the pool its warps find first; an item is a
// row's K head or V head.
template <typename T, int HD, bool VEC, int ROWS>
__global__ void __launch_bounds__(kThreads, 3) paged_append_kernel(const AppendParams p) {
  constexpr int kLanes = HD / 16, kHalf = HD / 2, kItems = kThreads / kLanes;
  constexpr int kBatch = 2;
  __shared__ Turns<HD> cs[ROWS];
  __shared__ long long place[ROWS];                        // pool row of KV head 0, or -1
  __shared__ int position[ROWS];
  const int row0 = blockIdx.x * ROWS, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = tid % kLanes;
  const int heads = 2 * p.pv.n_kv, items = min(ROWS, p.n_rows - row0) * heads;
  pdl_wait();
  pdl_trigger();
  auto load = [&](int i, Eight<T>& a, Eight<T>& b) {
    const int r = p.by_heads(i), h = i - r * heads;
    const bool is_k = h < p.pv.n_kv;
    const T* src = static_cast<const T*>(is_k ? p.k : p.v) + (row0 + r) * p.kv_ld +
                   (long long)(is_k ? h : h - p.pv.n_kv) * HD + 8 * sub;
    a.template load<VEC>(src);
    b.template load<VEC>(src + kHalf);
  };
  for (int i0 = 0; i0 < items; i0 += kBatch * kItems) {    // block-uniform
    Eight<T> a[kBatch], b[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kItems + tid / kLanes;
      if (i < items) load(i, a[k], b[k]);
    }
    if (i0 == 0) {
      for (int r = warp; r < ROWS; r += kThreads / 32) {
        const int row = row0 + r;
        long long at = -1;
        int pos = 0;
        if (row < p.n_rows) {
          const int req = request_of(p.row_off, p.n_req, row, lane);
          if (req < p.n_req && row >= p.row_off[req]) {
            const int slot = p.pos0[req] + (row - p.row_off[req]);
            pos = p.pos ? p.pos[row] : slot;
            const int page = pos < 0 ? -1 : page_of(p.pv, req, slot);
            if (page >= 0) at = pool_row(p.pv, page, 0, slot);
          }
        }
        if (lane == 0) {
          place[r] = at;
          position[r] = pos;
        }
      }
      __syncthreads();
      if (p.rotate) {
        for (int i = tid; i < ROWS * kHalf; i += kThreads)
          cs[i / kHalf].put(i % kHalf, turn_cs(position[i / kHalf], p.fr.f[i % kHalf]));
        __syncthreads();
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kItems + tid / kLanes, r = p.by_heads(i), h = i - r * heads;
      if (i >= items || place[r] < 0) continue;
      const bool is_k = h < p.pv.n_kv;
      if (is_k && p.rotate) {
        float2 x[4], y[4];
        a[k].get(x);
        b[k].get(y);
        cs[r].rotate(x, y, sub);
        a[k].set(x);
        b[k].set(y);
      }
      const long long row = place[r] + ((long long)(is_k ? h : h - p.pv.n_kv) << p.pv.page_shift);
      T* dst = static_cast<T*>(is_k ? p.pv.k : p.pv.v) + row * HD + 8 * sub;
      a[k].template store<true>(dst);
      b[k].template store<true>(dst + kHalf);
    }
  }
}

// ---------------------------------------------------------------------------
// The append into a cache held in 8 bits
// ---------------------------------------------------------------------------
// A scale belongs to a block of 16 slots, so a block is a CTA's, and a block of one KV
// head's keys or values a warp's: the warp holds all its rows in registers (16 rows of
// 128 elements are 64 to a lane), rotates them, finds the largest element and the
// scale, and writes the codes.  Memory bounds it: rows in once, codes and scales out.
// (A CTA of four warps: its block's rotations are formed, and its rows arrive, beside those of
// three others.  88 MB of prompt rows take 21.8 us, with eight warps 22.4; of fp32 without
// rotation 8.5 and 10.1.)
constexpr int kThreadsE4M3 = 128;

struct AppendE4M3Params {
  PagedView pv;
  uint8_t *k_scale, *v_scale;
  int n_req, n_rows;
  const int32_t *row_off, *pos0, *pos;
  const void *k, *v;
  long long kv_ld;
  int rotate;
  RopeTurns fr;
};

// Biased exponent of the smallest power of two >= 2^-127 at which `top` (finite, >= 0)
// is at most 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_for(float top) {
  const uint32_t b = __float_as_uint(top);
  return max(static_cast<int>(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0), 0);
}
// 2^(127 - b) for a biased exponent 0 <= b <= 254 (2^-127 is subnormal).
__device__ __forceinline__ float unscale(int b) {
  return __uint_as_float(b < kTopScale ? static_cast<uint32_t>(254 - b) << 23 : 0x00400000u);
}

__device__ __forceinline__ uint32_t codes4(float2 a, float2 b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3)) |
         static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
}
__device__ __forceinline__ float2 values2(uint32_t codes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3)));
}
// Four codes times f (a power of two below 1), rounded again.
__device__ __forceinline__ uint32_t recode4(uint32_t c, float f) {
  const float2 a = values2(c & 0xFFFFu), b = values2(c >> 16), f2 = make_float2(f, f);
  return codes4(__fmul2_rn(a, f2), __fmul2_rn(b, f2));
}

// Blocks of requests lie on a line without a prefix sum: those of request r, at most
// (n + 30) / 16 for its n rows, begin at row_off[r] / 16 + 2 r.
__device__ __forceinline__ int first_block(const AppendE4M3Params& p, int r) {
  return (min(max(__ldg(p.row_off + r), 0), p.n_rows) >> 4) + 2 * r;
}

template <typename T, int HD, bool VEC>
__global__ void __launch_bounds__(kThreadsE4M3, 3) paged_append_e4m3_kernel(const AppendE4M3Params p) {
  constexpr int kLanes = HD / 16, kHalf = HD / 2, kPass = 32 / kLanes, kPasses = kScaleBlock / kPass;
  __shared__ Turns<HD> cs[kScaleBlock];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % kLanes;
  pdl_wait();
  pdl_trigger();
  const int req = last_begun(p.n_req, lane, [&](int r) { return first_block(p, r) <= static_cast<int>(blockIdx.x); });
  const int row0 = min(max(p.row_off[req], 0), p.n_rows);
  const int n = min(max(p.row_off[req + 1], row0), p.n_rows) - row0, p0 = p.pos0[req];
  const long long s0 = ((long long)(p0 >> 4) + (static_cast<int>(blockIdx.x) - first_block(p, req))) * kScaleBlock;
  if (n == 0 || s0 >= (long long)p0 + n || s0 < 0 || s0 >= (1ll << 30)) return;    // block-uniform
  const int slot0 = static_cast<int>(s0);
  const int lead = row0 - p0 + slot0;                      // row of the block's first slot, were it new
  const int old = min(max(p0 - slot0, 0), kScaleBlock);    // slots that hold earlier tokens
  const int end = static_cast<int>(min((long long)p0 + n - slot0, (long long)kScaleBlock));

  // the slots whose rows are stored
  auto stored = [&](int s) { return s >= old && s < end && (!p.pos || __ldg(p.pos + lead + s) >= 0); };
  const uint32_t live = __ballot_sync(0xffffffffu, lane < kScaleBlock && stored(lane));
  if (live == 0) return;

  const int items = 2 * p.pv.n_kv, warps = gridDim.y * (kThreadsE4M3 / 32);
  Eight<T> a[kPasses], b[kPasses];
  auto load = [&](int h) {
    const bool is_k = h < p.pv.n_kv;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int s = i * kPass + lane / kLanes;
      if (!((live >> s) & 1u)) continue;
      const T* src = static_cast<const T*>(is_k ? p.k : p.v) + (lead + s) * p.kv_ld +
                     (long long)(is_k ? h : h - p.pv.n_kv) * HD + 8 * sub;
      a[i].template load<VEC>(src);
      b[i].template load<VEC>(src + kHalf);
    }
  };
  int h = blockIdx.y * (kThreadsE4M3 / 32) + warp;
  if (h < items) load(h);
  const int page = page_of(p.pv, req, slot0);              // (asked for beside the rows)
  if (page < 0) return;                                    // block-uniform
  if (p.rotate) {
    const uint64_t fr = p.fr.f[tid % kHalf];               // (lanes' own constants: asked for once)
    for (int s = tid / kHalf; s < kScaleBlock; s += kThreadsE4M3 / kHalf)
      if ((live >> s) & 1u) cs[s].put(tid % kHalf, turn_cs(p.pos ? __ldg(p.pos + lead + s) : slot0 + s, fr));
    __syncthreads();
  }
  for (; h < items; h += warps) {
    const bool is_k = h < p.pv.n_kv;
    const int g = is_k ? h : h - p.pv.n_kv;
    const long long row = pool_row(p.pv, page, g, slot0);
    uint8_t* scale = (is_k ? p.k_scale : p.v_scale) + row / kScaleBlock;
    const int was = old > 0 ? min(static_cast<int>(*scale), kTopScale) : 0;
    float2 x[kPasses][4], y[kPasses][4];
    float top = 0.f;                                       // (a maximum passes over NaN)
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int s = i * kPass + lane / kLanes;
      if (!((live >> s) & 1u)) continue;
      a[i].get(x[i]);
      b[i].get(y[i]);
      if (is_k && p.rotate) cs[s].rotate(x[i], y[i], sub);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        top = fmaxf(fmaxf(top, fabsf(x[i][j].x)), fabsf(x[i][j].y));
        top = fmaxf(fmaxf(top, fabsf(y[i][j].x)), fabsf(y[i][j].y));
      }
    }
    if (h + warps < items) load(h + warps);
    if (__any_sync(0xffffffffu, top > CUDART_MAX_NORMAL_F)) {      // (rare) infinities: NaN, and no maximum
      top = 0.f;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        if (!((live >> (i * kPass + lane / kLanes)) & 1u)) continue;
        auto see = [&](float& v) {
          if (!(fabsf(v) <= CUDART_MAX_NORMAL_F)) v = CUDART_NAN_F;
          top = fmaxf(top, fabsf(v));
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          see(x[i][j].x);
          see(x[i][j].y);
          see(y[i][j].x);
          see(y[i][j].y);
        }
      }
    }
    const int fits = scale_for(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))));
    const int now = max(fits, was);
    const float f = unscale(now);
    const float2 f2 = make_float2(f, f);
    uint8_t* dst = static_cast<uint8_t*>(is_k ? p.pv.k : p.pv.v) + row * HD;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int s = i * kPass + lane / kLanes;
      uint2* lo = reinterpret_cast<uint2*>(dst + s * HD + 8 * sub);
      uint2* hi = reinterpret_cast<uint2*>(dst + s * HD + kHalf + 8 * sub);
      if ((live >> s) & 1u) {
        *lo = make_uint2(codes4(__fmul2_rn(x[i][0], f2), __fmul2_rn(x[i][1], f2)),
                         codes4(__fmul2_rn(x[i][2], f2), __fmul2_rn(x[i][3], f2)));
        *hi = make_uint2(codes4(__fmul2_rn(y[i][0], f2), __fmul2_rn(y[i][1], f2)),
                         codes4(__fmul2_rn(y[i][2], f2), __fmul2_rn(y[i][3], f2)));
      } else if (s < old && now > was) {
        const float shift = __uint_as_float(static_cast<uint32_t>(127 - min(now - was, 64)) << 23);   // 2^(was - now)
        *lo = make_uint2(recode4(lo->x, shift), recode4(lo->y, shift));
        *hi = make_uint2(recode4(hi->x, shift), recode4(hi->y, shift));
      }
    }
    if (lane == 0) *scale = static_cast<uint8_t>(now);
  }
}

bool many(int rows) { return rows >= 6 * num_sms(); }

template <typename T, int HD, bool VEC>
void launch_norm_rope(const NormRopeParams& p, cudaStream_t st) {
  if (many(p.n_rows))
    launch_k(qk_norm_rope_kernel<T, HD, VEC, kNormRows>, dim3((p.n_rows + kNormRows - 1) / kNormRows),
             dim3(kThreads), 0, st, p);
  else
    launch_k(qk_norm_rope_kernel<T, HD, VEC, 1>, dim3(p.n_rows, 2), dim3(kThreads), 0, st, p);
}

template <typename T, int HD, bool VEC>
void launch_append(const AppendParams& p, cudaStream_t st) {
  if (many(p.n_rows))
    launch_k(paged_append_kernel<T, HD, VEC, kAppendRows>, dim3((p.n_rows + kAppendRows - 1) / kAppendRows),
             dim3(kThreads), 0, st, p);
  else
    launch_k(paged_append_kernel<T, HD, VEC, 1>, dim3(p.n_rows), dim3(kThreads), 0, st, p);
}

// One item to a warp where there are few blocks (latency), all of a block's to one CTA
// where there are many, which then forms the rotations once.  8 heads of 128, bf16, rotated,
// one CTA to a block / several, us: 66 blocks 6.8 / 4.2, 264 (128 single tokens) 7.0 / 6.8,
// 258 (a prompt of 4096) 8.3 / 10.4, 528 7.4 / 10.0, 1026 23.2 / 33.0; 2 heads of 64: the same.
template <typename T, int HD, bool VEC>
void launch_append_e4m3(const AppendE4M3Params& p, cudaStream_t st) {
  const int blocks = (p.n_rows >> 4) + 2 * p.n_req, per = kThreadsE4M3 / 32;
  const int split = 2 * blocks >= 3 * num_sms() ? 1 : (2 * p.pv.n_kv + per - 1) / per;
  launch_k(paged_append_e4m3_kernel<T, HD, VEC>, dim3(blocks, split), dim3(kThreadsE4M3), 0, st, p);
}

bool aligned16(const void* p, long long ld_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld_bytes)) & 15) == 0;
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

dflash_status dflash_qk_norm_rope(int n_rows, int n_q, int n_kv, int head_dim, int dtype,
                                  const void* q_gain, const void* k_gain, float eps, float theta,
                                  const int32_t* pos, const void* q, long long q_ld,
                                  const void* k, long long k_ld, void* q_out,
                                  long long q_out_ld, void* k_out, long long k_out_ld,
                                  void* stream) {
  DFL_REQUIRE(n_rows >= 0 && n_q >= 0 && n_kv >= 0, "qk norm rope: sizes must be >= 0");
  DFL_REQUIRE(n_q <= kMaxHeads && n_kv <= kMaxHeads, "qk norm rope: more than %d heads", kMaxHeads);
  DFL_REQUIRE(head_dim == 64 || head_dim == 128, "qk norm rope: head_dim must be 64 or 128");
  DFL_REQUIRE(dtype == DFLASH_F32 || dtype == DFLASH_BF16, "qk norm rope: dtype must be F32 or BF16");
  DFL_REQUIRE(eps >= 0.f && eps < 1e30f, "qk norm rope: eps must be >= 0");
  DFL_REQUIRE(theta == 0.f || (theta > 0.f && theta < 1e30f),
              "qk norm rope: theta must be 0 (no rotation) or positive");
  const long long qw = (long long)n_q * head_dim, kw = (long long)n_kv * head_dim;
  DFL_REQUIRE(n_q == 0 || (q_ld >= qw && q_out_ld >= qw), "qk norm rope: query row stride too small");
  DFL_REQUIRE(n_kv == 0 || (k_ld >= kw && k_out_ld >= kw), "qk norm rope: key row stride too small");
  if (n_rows == 0 || n_q + n_kv == 0) return DFLASH_OK;
  DFL_REQUIRE((n_q == 0 || (q && q_out)) && (n_kv == 0 || (k && k_out)) && (theta == 0.f || pos),
              "qk norm rope: null pointer argument");
  DFL_REQUIRE((n_q == 0 || q != q_out || q_ld == q_out_ld) &&
                  (n_kv == 0 || k != k_out || k_ld == k_out_ld),
              "qk norm rope: in place needs the same row stride");
  NormRopeParams p{};
  p.n_rows = n_rows;
  p.by_q = divide_by(n_q > 0 ? n_q : 1);
  p.by_kv = divide_by(n_kv > 0 ? n_kv : 1);
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.q_gain = q_gain;
  p.k_gain = k_gain;
  p.eps = eps;
  p.rotate = theta > 0.f;
  if (p.rotate) p.fr = rope_turns(theta, head_dim);
  p.pos = pos;
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_ld = q_ld;
  p.k_ld = k_ld;
  p.q_out_ld = q_out_ld;
  p.k_out_ld = k_out_ld;
  const long long es = dtype == DFLASH_F32 ? 4 : 2;
  const bool vec = aligned16(q_gain, 0) && aligned16(k_gain, 0) &&
                   (n_q == 0 || (aligned16(q, q_ld * es) && aligned16(q_out, q_out_ld * es))) &&
                   (n_kv == 0 || (aligned16(k, k_ld * es) && aligned16(k_out, k_out_ld * es)));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope ts("qk_norm_rope", st);
    auto go = [&](auto t) {
      using T = decltype(t);
      if (head_dim == 128)
        vec ? launch_norm_rope<T, 128, true>(p, st) : launch_norm_rope<T, 128, false>(p, st);
      else
        vec ? launch_norm_rope<T, 64, true>(p, st) : launch_norm_rope<T, 64, false>(p, st);
    };
    dtype == DFLASH_BF16 ? go(__nv_bfloat16()) : go(float());
  }
  return check_launch("qk norm rope");
}

dflash_status dflash_paged_append(const dflash_pages* pages, int n_req, int n_rows,
                                  const int32_t* row_off, const int32_t* pos0,
                                  const int32_t* pos, const void* k, const void* v,
                                  long long kv_ld, float theta, void* stream) {
  AppendParams p{};
  const dflash_status s = check_pages(pages, n_req, "paged append", &p.pv);
  if (s) return s;
  DFL_REQUIRE(n_req >= 0 && n_rows >= 0, "paged append: sizes must be >= 0");
  DFL_REQUIRE(2 * (long long)pages->n_kv <= kMaxHeads, "paged append: more than %d KV heads", kMaxHeads / 2);
  DFL_REQUIRE(kv_ld >= (long long)pages->n_kv * pages->head_dim, "paged append: row stride too small");
  DFL_REQUIRE(theta == 0.f || (theta > 0.f && theta < 1e30f),
              "paged append: theta must be 0 (no rotation) or positive");
  if (n_req == 0 || n_rows == 0) return DFLASH_OK;
  DFL_REQUIRE(row_off && pos0 && k && v, "paged append: null pointer argument");
  p.n_req = n_req;
  p.n_rows = n_rows;
  p.by_heads = divide_by(2 * pages->n_kv);
  p.row_off = row_off;
  p.pos0 = pos0;
  p.pos = pos;
  p.k = k;
  p.v = v;
  p.kv_ld = kv_ld;
  p.rotate = theta > 0.f;
  if (p.rotate) p.fr = rope_turns(theta, pages->head_dim);
  const long long es = pages->dtype == DFLASH_F32 ? 4 : 2;
  const bool vec = aligned16(k, kv_ld * es) && aligned16(v, kv_ld * es);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope ts("paged_append", st);
    auto go = [&](auto t) {
      using T = decltype(t);
      if (pages->head_dim == 128)
        vec ? launch_append<T, 128, true>(p, st) : launch_append<T, 128, false>(p, st);
      else
        vec ? launch_append<T, 64, true>(p, st) : launch_append<T, 64, false>(p, st);
    };
    pages->dtype == DFLASH_BF16 ? go(__nv_bfloat16()) : go(float());
  }
  return check_launch("paged append");
}

dflash_status dflash_paged_append_e4m3(const dflash_pages_e4m3* pages, int n_req, int n_rows,
                                       const int32_t* row_off, const int32_t* pos0,
                                       const int32_t* pos, int dtype, const void* k,
                                       const void* v, long long kv_ld, float theta, void* stream) {
  AppendE4M3Params p{};
  const dflash_status s = check_pages(pages, n_req, "paged append e4m3", &p.pv);
  if (s) return s;
  DFL_REQUIRE(n_req >= 0 && n_rows >= 0, "paged append e4m3: sizes must be >= 0");
  DFL_REQUIRE((n_rows >> 4) + 2 * (long long)n_req < (1ll << 30), "paged append e4m3: too many rows and requests");
  DFL_REQUIRE(dtype == DFLASH_F32 || dtype == DFLASH_BF16, "paged append e4m3: dtype must be F32 or BF16");
  DFL_REQUIRE(2 * (long long)pages->n_kv <= kMaxHeads, "paged append e4m3: more than %d KV heads", kMaxHeads / 2);
  DFL_REQUIRE(kv_ld >= (long long)pages->n_kv * pages->head_dim, "paged append e4m3: row stride too small");
  DFL_REQUIRE(theta == 0.f || (theta > 0.f && theta < 1e30f),
              "paged append e4m3: theta must be 0 (no rotation) or positive");
  if (n_req == 0 || n_rows == 0) return DFLASH_OK;
  DFL_REQUIRE(row_off && pos0 && k && v, "paged append e4m3: null pointer argument");
  p.k_scale = pages->k_scale;
  p.v_scale = pages->v_scale;
  p.n_req = n_req;
  p.n_rows = n_rows;
  p.row_off = row_off;
  p.pos0 = pos0;
  p.pos = pos;
  p.k = k;
  p.v = v;
  p.kv_ld = kv_ld;
  p.rotate = theta > 0.f;
  if (p.rotate) p.fr = rope_turns(theta, pages->head_dim);
  const long long es = dtype == DFLASH_F32 ? 4 : 2;
  const bool vec = aligned16(k, kv_ld * es) && aligned16(v, kv_ld * es);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope ts("paged_append_e4m3", st);
    auto go = [&](auto t) {
      using T = decltype(t);
      if (pages->head_dim == 128)
        vec ? launch_append_e4m3<T, 128, true>(p, st) : launch_append_e4m3<T, 128, false>(p, st);
      else
        vec ? launch_append_e4m3<T, 64, true>(p, st) : launch_append_e4m3<T, 64, false>(p, st);
    };
    dtype == DFLASH_BF16 ? go(__nv_bfloat16()) : go(float());
  }
  return check_launch("paged append e4m3");
}

}  // extern "C"
