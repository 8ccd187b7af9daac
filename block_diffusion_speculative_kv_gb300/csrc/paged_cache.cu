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
// over them.  A row's cosines and sines (64-bit angles, rope_cs) are formed
// once by the CTA and shared by all its heads, while the loads are in flight.
#include "kernels.h"
#include "paged.cuh"

namespace dfl {

dflash_status check_pages(const dflash_pages* p, const char* what, PagedView* out) {
  DFL_REQUIRE(p, "%s: null pages", what);
  DFL_REQUIRE(p->dtype == DFLASH_F32 || p->dtype == DFLASH_BF16, "%s: dtype must be F32 or BF16",
              what);
  DFL_REQUIRE(p->head_dim == 64 || p->head_dim == 128, "%s: head_dim must be 64 or 128", what);
  DFL_REQUIRE(p->page_size >= 16 && p->page_size <= 1024 &&
                  (p->page_size & (p->page_size - 1)) == 0,
              "%s: page_size must be a power of two in [16, 1024]", what);
  DFL_REQUIRE(p->n_kv >= 1 && p->n_pages >= 1 && p->table_ld >= 1,
              "%s: need n_kv, n_pages and table_ld >= 1", what);
  DFL_REQUIRE((long long)p->table_ld * p->page_size < (1ll << 31),
              "%s: a request's slots exceed 2^31", what);
  DFL_REQUIRE((long long)p->n_pages * p->n_kv * p->page_size < (1ll << 31),
              "%s: the pool's rows exceed 2^31", what);
  DFL_REQUIRE(p->k && p->v && p->table, "%s: null pool or table", what);
  DFL_REQUIRE(((reinterpret_cast<uintptr_t>(p->k) | reinterpret_cast<uintptr_t>(p->v)) & 15) == 0,
              "%s: pools must be 16-byte aligned", what);
  *out = PagedView{p->k, p->v, p->table, p->table_ld, p->n_pages, log2_int(p->page_size), p->n_kv};
  return DFLASH_OK;
}

namespace {

// Eight consecutive elements as fp32; VEC: the address is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (VEC && sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else if constexpr (VEC) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32<T>(p[i]);
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (VEC && sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if constexpr (VEC) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = from_f32<T>(x[i]);
  }
}

__device__ __forceinline__ void rotate8(float (&a)[8], float (&b)[8], const float2* cs) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 c = cs[i];
    const float x = a[i], y = b[i];
    a[i] = x * c.x - y * c.y;
    b[i] = y * c.x + x * c.y;
  }
}

struct NormRopeParams {
  int n_q, n_kv;
  const void *q_gain, *k_gain;
  float eps;
  int rotate;
  RopeFreqs fr;
  const int32_t* pos;
  const void *q, *k;
  void *q_out, *k_out;
  long long q_ld, k_ld, q_out_ld, k_out_ld;
};

// One CTA per row.  Lanes of a head: HD / 16, so a warp's shuffle groups never
// straddle heads; the block is a whole number of warps and idle lanes take part
// in the shuffles.
template <typename T, int HD, bool VEC>
__global__ void qk_norm_rope_kernel(const NormRopeParams p) {
  constexpr int kLanes = HD / 16, kHalf = HD / 2;
  __shared__ float2 cs[kHalf];
  const int row = blockIdx.x, tid = threadIdx.x;
  const int sub = tid % kLanes, heads = p.n_q + p.n_kv;
  pdl_wait();
  pdl_trigger();
  const int pos = p.pos ? p.pos[row] : 0;
  if (pos < 0) return;
  for (int h0 = 0; h0 < heads; h0 += blockDim.x / kLanes) {
    const int h = h0 + tid / kLanes;
    const bool live = h < heads, is_q = h < p.n_q;
    const T* src = nullptr;
    T* dst = nullptr;
    if (live) {
      const long long col = (long long)(is_q ? h : h - p.n_q) * HD + 8 * sub;
      src = static_cast<const T*>(is_q ? p.q : p.k) + row * (is_q ? p.q_ld : p.k_ld) + col;
      dst = static_cast<T*>(is_q ? p.q_out : p.k_out) + row * (is_q ? p.q_out_ld : p.k_out_ld) + col;
    }
    float a[8] = {}, b[8] = {};
    if (live) {
      load8<T, VEC>(src, a);
      load8<T, VEC>(src + kHalf, b);
    }
    if (h0 == 0 && p.rotate) {
      for (int i = tid; i < kHalf; i += blockDim.x) cs[i] = rope_cs(pos, i, p.fr);
      __syncthreads();
    }
    const T* gain = static_cast<const T*>(is_q ? p.q_gain : p.k_gain);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
#pragma unroll
    for (int off = kLanes / 2; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (!live) continue;
    if (gain) {
      const float inv = 1.f / sqrtf(ss * (1.f / HD) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= inv * to_f32<T>(gain[8 * sub + i]);
        b[i] *= inv * to_f32<T>(gain[kHalf + 8 * sub + i]);
      }
    }
    if (p.rotate) rotate8(a, b, cs + 8 * sub);
    store8<T, VEC>(dst, a);
    store8<T, VEC>(dst + kHalf, b);
  }
}

struct AppendParams {
  PagedView pv;
  int n_req, n_rows;
  const int32_t *row_off, *pos0, *pos;
  const void *k, *v;
  long long kv_ld;
  int rotate;
  RopeFreqs fr;
};

// One CTA per row: K's heads, then V's, HD / 16 lanes each.
template <typename T, int HD, bool VEC>
__global__ void paged_append_kernel(const AppendParams p) {
  constexpr int kLanes = HD / 16, kHalf = HD / 2;
  __shared__ float2 cs[kHalf];
  const int row = blockIdx.x, tid = threadIdx.x, sub = tid % kLanes;
  pdl_wait();
  pdl_trigger();
  const int req = request_of(p.row_off, p.n_req, row, tid & 31);
  if (req >= p.n_req || row < p.row_off[req]) return;
  const int slot = p.pos0[req] + (row - p.row_off[req]);
  const int pos = p.pos ? p.pos[row] : slot;
  if (pos < 0) return;
  const int page = page_of(p.pv, req, slot);
  if (page < 0) return;
  for (int h0 = 0; h0 < 2 * p.pv.n_kv; h0 += blockDim.x / kLanes) {
    const int h = h0 + tid / kLanes;
    const bool live = h < 2 * p.pv.n_kv, is_k = h < p.pv.n_kv;
    const int g = is_k ? h : h - p.pv.n_kv;
    float a[8] = {}, b[8] = {};
    if (live) {
      const T* src = static_cast<const T*>(is_k ? p.k : p.v) + row * p.kv_ld + (long long)g * HD + 8 * sub;
      load8<T, VEC>(src, a);
      load8<T, VEC>(src + kHalf, b);
    }
    if (h0 == 0 && p.rotate) {
      for (int i = tid; i < kHalf; i += blockDim.x) cs[i] = rope_cs(pos, i, p.fr);
      __syncthreads();
    }
    if (!live) continue;
    if (is_k && p.rotate) rotate8(a, b, cs + 8 * sub);
    T* dst = static_cast<T*>(is_k ? p.pv.k : p.pv.v) + pool_row(p.pv, page, g, slot) * HD + 8 * sub;
    store8<T, true>(dst, a);
    store8<T, true>(dst + kHalf, b);
  }
}

template <typename T, int HD>
void launch_norm_rope(const NormRopeParams& p, int n_rows, bool vec, cudaStream_t st) {
  const int lanes = (p.n_q + p.n_kv) * (HD / 16);
  const int threads = lanes < 512 ? (lanes + 31) / 32 * 32 : 512;
  if (vec)
    launch_k(qk_norm_rope_kernel<T, HD, true>, dim3(n_rows), dim3(threads), 0, st, p);
  else
    launch_k(qk_norm_rope_kernel<T, HD, false>, dim3(n_rows), dim3(threads), 0, st, p);
}

template <typename T, int HD>
void launch_append(const AppendParams& p, bool vec, cudaStream_t st) {
  const int lanes = 2 * p.pv.n_kv * (HD / 16);
  const int threads = lanes < 512 ? (lanes + 31) / 32 * 32 : 512;
  if (vec)
    launch_k(paged_append_kernel<T, HD, true>, dim3(p.n_rows), dim3(threads), 0, st, p);
  else
    launch_k(paged_append_kernel<T, HD, false>, dim3(p.n_rows), dim3(threads), 0, st, p);
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
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.q_gain = q_gain;
  p.k_gain = k_gain;
  p.eps = eps;
  p.rotate = theta > 0.f;
  if (p.rotate) p.fr = rope_freqs(theta, head_dim);
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
  const bool vec = (n_q == 0 || (aligned16(q, q_ld * es) && aligned16(q_out, q_out_ld * es))) &&
                   (n_kv == 0 || (aligned16(k, k_ld * es) && aligned16(k_out, k_out_ld * es)));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope ts("qk_norm_rope", st);
    if (dtype == DFLASH_BF16)
      head_dim == 128 ? launch_norm_rope<__nv_bfloat16, 128>(p, n_rows, vec, st)
                      : launch_norm_rope<__nv_bfloat16, 64>(p, n_rows, vec, st);
    else
      head_dim == 128 ? launch_norm_rope<float, 128>(p, n_rows, vec, st)
                      : launch_norm_rope<float, 64>(p, n_rows, vec, st);
  }
  return check_launch("qk norm rope");
}

dflash_status dflash_paged_append(const dflash_pages* pages, int n_req, int n_rows,
                                  const int32_t* row_off, const int32_t* pos0,
                                  const int32_t* pos, const void* k, const void* v,
                                  long long kv_ld, float theta, void* stream) {
  AppendParams p{};
  const dflash_status s = check_pages(pages, "paged append", &p.pv);
  if (s) return s;
  DFL_REQUIRE(n_req >= 0 && n_rows >= 0, "paged append: sizes must be >= 0");
  DFL_REQUIRE(kv_ld >= (long long)pages->n_kv * pages->head_dim, "paged append: row stride too small");
  DFL_REQUIRE(theta == 0.f || (theta > 0.f && theta < 1e30f),
              "paged append: theta must be 0 (no rotation) or positive");
  if (n_req == 0 || n_rows == 0) return DFLASH_OK;
  DFL_REQUIRE(row_off && pos0 && k && v, "paged append: null pointer argument");
  p.n_req = n_req;
  p.n_rows = n_rows;
  p.row_off = row_off;
  p.pos0 = pos0;
  p.pos = pos;
  p.k = k;
  p.v = v;
  p.kv_ld = kv_ld;
  p.rotate = theta > 0.f;
  if (p.rotate) p.fr = rope_freqs(theta, pages->head_dim);
  const long long es = pages->dtype == DFLASH_F32 ? 4 : 2;
  const bool vec = aligned16(k, kv_ld * es) && aligned16(v, kv_ld * es);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope ts("paged_append", st);
    if (pages->dtype == DFLASH_BF16)
      pages->head_dim == 128 ? launch_append<__nv_bfloat16, 128>(p, vec, st)
                             : launch_append<__nv_bfloat16, 64>(p, vec, st);
    else
      pages->head_dim == 128 ? launch_append<float, 128>(p, vec, st)
                             : launch_append<float, 64>(p, vec, st);
  }
  return check_launch("paged append");
}

}  // extern "C"
