// Logits before sampling: bias, penalties for repeated tokens, allowed tokens.
//
// "Accelerating Speculative Decoding with Block Diffusion Draft Trees", section
// 3.4.5: the target's choice at a tree node is made as if its path had been
// generated, so a penalty at a node counts the node's ancestors too.  Per row with
// past tokens (history, then its path) and per token v:
//
//   y = l_v + bias_v,  y = y > 0 ? y / rho : y rho          if v occurred,
//   y = y - phi c - pi   for the c > 0 times it was generated,  -inf if not allowed.
//
// HBM bounds it: logits in once, out once (a bit more for each token with a grammar).
// A CTA takes one stretch of the vocabulary for several rows of one request: it counts
// the request's history in that stretch once, in shared memory, and from row to row
// adds and takes away the tokens by which their paths differ.  A bit for each token
// says whether it occurred or has a bias at all; most 16-byte pieces have none and are
// only copied.
#include <math_constants.h>

#include "common.cuh"

namespace dfl {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxVocab = 1 << 22;

struct AdjustParams {
  int n_req, rows, vocab;
  const void* logits;
  void* out;
  long long ld, out_ld;
  const int32_t* row_off;
  const int32_t* history;
  int history_ld;
  const int32_t *history_len, *prompt_len;
  const float *repetition, *presence, *frequency;
  const int32_t* tok;
  const uint32_t* mask;
  int mask_ld;
  const int32_t* bias_tok;
  const float* bias_val;
  int n_bias;
  const uint32_t* allowed;
  long long allowed_ld;
};

// 16 bytes of a row as fp32.
template <typename T>
struct Piece {
  static constexpr int V = 16 / sizeof(T);
  float v[V];
  __device__ __forceinline__ void get(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ uint4 set() const {
    uint32_t w[4];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Groups of ROWS rows lie on a line without a prefix sum: those of request r begin at
// row_off[r] / ROWS + r.
template <int ROWS>
__device__ __forceinline__ int first_group(const AdjustParams& p, int r) {
  return min(max(__ldg(p.row_off + r), 0), p.rows) / ROWS + r;
}

template <typename T, int C, int ROWS>
__global__ void __launch_bounds__(kThreads) logits_adjust_kernel(const AdjustParams p) {
  constexpr int V = Piece<T>::V, kN = C / V / kThreads;    // pieces of a row to a thread, and one more
  static_assert(C % (V * kThreads) == 0);
  __shared__ uint32_t sCount[C];                           // times generated; the top bit: in the prompt
  __shared__ uint32_t sBias[C];                            // 1 + place in the list of biases
  __shared__ uint32_t sSome[C / 32 + 1];                   // tokens that may have changed
  const int tid = threadIdx.x, lane = tid & 31, c0 = blockIdx.y * C, c1 = min(c0 + C, p.vocab);
  pdl_wait();
  pdl_trigger();
  const int group = blockIdx.x;
  const int req = last_begun(p.n_req, lane, [&](int r) { return first_group<ROWS>(p, r) <= group; });
  const int row0 = min(max(p.row_off[req], 0), p.rows);
  const int n = min(max(p.row_off[req + 1], row0), p.rows) - row0;
  const int i0 = (group - first_group<ROWS>(p, req)) * ROWS, i1 = min(i0 + ROWS, n);
  if (i0 >= i1) return;                                    // block-uniform
  const float rho = p.repetition ? __ldg(p.repetition + req) : 1.f;
  const float phi = p.frequency ? __ldg(p.frequency + req) : 0.f;
  const float pi = p.presence ? __ldg(p.presence + req) : 0.f;
  const bool track = rho != 1.f || phi != 0.f || pi != 0.f;
  const bool change = track || p.n_bias > 0;

  auto note = [&](int t) { atomicOr(&sSome[t >> 5], 1u << (t & 31)); };
  auto path = [&](int j, int by) {                         // the request's row j joins the past, or leaves it
    const int t = __ldg(p.tok + row0 + j) - c0;
    if (static_cast<unsigned>(t) >= static_cast<unsigned>(c1 - c0)) return;
    atomicAdd(&sCount[t], static_cast<uint32_t>(by));
    if (by > 0) note(t);
  };
  const int words = p.mask ? min(p.mask_ld, (n + 31) / 32) : 0;
  auto sees = [&](int i, int j) {
    return (j >> 5) < words && ((__ldg(p.mask + (size_t)(row0 + i) * p.mask_ld + (j >> 5)) >> (j & 31)) & 1u);
  };

  if (change) {
    for (int t = tid; t < C; t += kThreads) {
      sCount[t] = 0;
      sBias[t] = 0;
    }
    if (tid <= C / 32) sSome[tid] = 0;
    __syncthreads();
    if (track) {
      const int len = p.history ? min(max(__ldg(p.history_len + req), 0), p.history_ld) : 0;
      const int prompt = p.prompt_len ? __ldg(p.prompt_len + req) : 0;
      const int32_t* h = p.history + (size_t)req * p.history_ld;
#pragma unroll 8
      for (int i = tid; i < len; i += kThreads) {
        const int t = __ldg(h + i) - c0;
        if (static_cast<unsigned>(t) >= static_cast<unsigned>(c1 - c0)) continue;
        i < prompt ? atomicOr(&sCount[t], 0x80000000u) : atomicAdd(&sCount[t], 1u);
        note(t);
      }
      if (p.tok && !p.mask)                                // the rows before this group
        for (int j = tid; j < i0; j += kThreads) path(j, 1);
    }
    for (int j = tid; j < p.n_bias; j += kThreads) {
      const int t = __ldg(p.bias_tok + (size_t)req * p.n_bias + j) - c0;
      if (static_cast<unsigned>(t) >= static_cast<unsigned>(c1 - c0)) continue;
      atomicMax(&sBias[t], static_cast<uint32_t>(j + 1));
      note(t);
    }
  }

  auto fix = [&](float y, int t) {
    const uint32_t count = sCount[t], b = sBias[t];
    if (b) y += __ldg(p.bias_val + (size_t)req * p.n_bias + b - 1);
    if (count) y = y > 0.f ? y / rho : y * rho;
    const uint32_t c = count & 0x7FFFFFFFu;
    if (c) y = y - phi * static_cast<float>(c) - pi;
    return y;
  };

  for (int i = i0; i < i1; ++i) {
    const long long row = row0 + i;
    const T* in = static_cast<const T*>(p.logits) + row * p.ld;
    T* out = static_cast<T*>(p.out) + row * p.out_ld;
    // pieces lie on 16-byte boundaries of the row; the first may begin before the stretch
    const int off_in = static_cast<int>(reinterpret_cast<uintptr_t>(in) / sizeof(T)) & (V - 1);
    const bool same = (static_cast<int>(reinterpret_cast<uintptr_t>(out) / sizeof(T)) & (V - 1)) == off_in;
    const int t0 = (c0 + off_in) / V * V - off_in;
    uint4 u[kN + 1];
#pragma unroll
    for (int k = 0; k <= kN; ++k) {
      const int t = t0 + (tid + k * kThreads) * V;
      if (t >= c1) continue;
      if (t >= c0 && t + V <= c1) {
        u[k] = *reinterpret_cast<const uint4*>(in + t);
      } else {
        __align__(16) T e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = t + j >= c0 && t + j < c1 ? in[t + j] : T(0.f);
        u[k] = *reinterpret_cast<const uint4*>(e);
      }
    }
    if (track && p.tok) {
      if (p.mask) {
        for (int j = tid; j < n; j += kThreads) {
          const bool now = sees(i, j), was = i > i0 && sees(i - 1, j);
          if (now != was) path(j, now ? 1 : -1);
        }
      } else if (tid == 0) {
        path(i, 1);
      }
    }
    if (change) __syncthreads();
    const uint32_t* allowed = p.allowed ? p.allowed + row * p.allowed_ld : nullptr;
#pragma unroll
    for (int k = 0; k <= kN; ++k) {
      const int t = t0 + (tid + k * kThreads) * V;
      if (t >= c1) continue;
      const bool full = t >= c0 && t + V <= c1;
      uint32_t may = 0xFFFFFFFFu, some = 0;                // a bit to an element
      if (allowed) {
        const int w = t >> 5, last = (p.vocab - 1) >> 5;
        const uint32_t lo = w >= 0 ? __ldg(allowed + w) : 0u;
        const uint32_t hi = (t & 31) + V > 32 && w < last ? __ldg(allowed + w + 1) : 0u;
        may = __funnelshift_r(lo, hi, t & 31);
      }
      if (change) {
        const int a = t - c0, w = a >> 5;                  // (a > -V: the word before the first has no bit)
        some = __funnelshift_r(w >= 0 ? sSome[w] : 0u, sSome[w + 1], a & 31);
      }
      Piece<T> x;
      x.get(u[k]);
      if (some & ((1u << V) - 1u)) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if ((some >> j) & 1u) x.v[j] = fix(x.v[j], t - c0 + j);
      }
      if ((may & ((1u << V) - 1u)) != (1u << V) - 1u) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (!((may >> j) & 1u)) x.v[j] = -CUDART_INF_F;
      }
      if (full && same) {
        *reinterpret_cast<uint4*>(out + t) = x.set();
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (t + j >= c0 && t + j < c1) out[t + j] = from_f32<T>(x.v[j]);
      }
    }
    if (change && i + 1 < i1) __syncthreads();             // the counts change for the next row
  }
}

template <typename T, int C, int ROWS>
void launch(const AdjustParams& p, cudaStream_t st) {
  const int groups = p.rows / ROWS + p.n_req;
  launch_k(logits_adjust_kernel<T, C, ROWS>, dim3(groups, (p.vocab + C - 1) / C), dim3(kThreads), 0, st, p);
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_logits_adjust(
    int n_req, int rows, int vocab, int dtype, const void* logits, long long ld, void* out, long long out_ld,
    const int32_t* row_off, const int32_t* history, int history_ld, const int32_t* history_len,
    const int32_t* prompt_len, const float* repetition, const float* presence, const float* frequency,
    const int32_t* tok, const uint32_t* mask, int mask_ld, const int32_t* bias_tok, const float* bias_val, int n_bias,
    const uint32_t* allowed, long long allowed_ld, void* stream) {
  DFL_REQUIRE(n_req >= 0 && rows >= 0, "logits adjust: sizes must be >= 0");
  DFL_REQUIRE(rows + (long long)n_req < (1ll << 30), "logits adjust: too many rows and requests");
  DFL_REQUIRE(vocab >= 1 && vocab <= kMaxVocab, "logits adjust: vocab must be in [1, %d]", kMaxVocab);
  DFL_REQUIRE(dtype == DFLASH_F32 || dtype == DFLASH_BF16, "logits adjust: dtype must be F32 or BF16");
  DFL_REQUIRE(ld >= vocab && out_ld >= vocab, "logits adjust: row strides smaller than vocab");
  DFL_REQUIRE(history == nullptr || (history_ld >= 1 && history_len), "logits adjust: history needs lengths");
  DFL_REQUIRE(mask == nullptr || (mask_ld >= 1 && tok), "logits adjust: a mask needs words and tokens");
  DFL_REQUIRE(n_bias >= 0 && n_bias <= (1 << 20), "logits adjust: n_bias must be in [0, 2^20]");
  DFL_REQUIRE(n_bias == 0 || (bias_tok && bias_val), "logits adjust: null bias list");
  DFL_REQUIRE(allowed == nullptr || allowed_ld * 32 >= vocab, "logits adjust: allowed rows shorter than vocab");
  if (n_req == 0 || rows == 0) return DFLASH_OK;
  DFL_REQUIRE(logits && out && row_off, "logits adjust: null pointer argument");
  DFL_REQUIRE(logits != out || ld == out_ld, "logits adjust: in place needs the same row stride");
  const size_t es = dtype == DFLASH_F32 ? 4 : 2;
  DFL_REQUIRE(((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out)) & (es - 1)) == 0,
              "logits adjust: logits and out must be aligned to their elements");
  const AdjustParams p = {n_req,    rows,       vocab,       logits,     out,        ld,       out_ld,    row_off,
                          history,  history_ld, history_len, prompt_len, repetition, presence, frequency, tok,
                          mask,     mask_ld,    bias_tok,    bias_val,   n_bias,     allowed,  allowed_ld};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope ts("logits_adjust", st);
    const bool few = (rows / 16 + n_req) * (long long)((vocab + 4095) / 4096) < 2 * num_sms();
    if (dtype == DFLASH_BF16)
      few ? launch<__nv_bfloat16, 2048, 4>(p, st) : launch<__nv_bfloat16, 4096, 16>(p, st);
    else
      few ? launch<float, 1024, 4>(p, st) : launch<float, 4096, 16>(p, st);
  }
  return check_launch("logits adjust");
}
