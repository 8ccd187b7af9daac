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
// the request's history in that stretch once, in shared memory, makes a sorted list of
// the tokens that occurred or have a bias, and lists the rows' own tokens that lie there.
// Then every warp works for itself, without another barrier: it brings a part of a row, 1, 2 or
// 4 KB (kDeep 2, 4, 8), picks from the list what the row's path holds, changes the listed tokens,
// a lane to a token, in a buffer of its own, and writes the part.  A history of 8192 tokens touches
// one token in 35, one of almost every 128 neighbours: changed where they are, in the
// registers of the lanes that have them, they made the warps' instructions the limit (480
// bf16 rows of 151936: 159 us).  Now those take 76 us by 2 KB (4.0 TB/s; a copy 46), 257 fp32 nodes
// of a tree 56 by 4 KB (5.6 TB/s), where waiting for rows bounds them; 256 bf16 requests of one
// row after 2048 tokens each 83 by 1 KB, half of that the histories' instructions.
//
// Each stretch of each group of rows goes through its request's history, so time grows with
// history times vocabulary.  Histories of 0 / 8192 / 32768 / 131072 tokens, us, bf16: 32 requests
// of 15 rows 56 / 72 / 109 / 230, 256 of one row 63 / 113 / 234 / 757, one row 6 / 12 / 23 / 63,
// one request of 257 rows 33 / 44 / 62 / 125: past about 30000 tokens they decide.
#include <math_constants.h>

#include "common.cuh"

namespace dfl {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxVocab = 1 << 22;
constexpr int kMaxHistory = 1 << 30;   // (steps past a history's end do not pass 2^31)

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

template <typename T>
struct Piece {                    // 16 bytes of a row
  static constexpr int V = 16 / sizeof(T);
};

// Groups of ROWS rows lie on a line without a prefix sum: those of request r begin at
// row_off[r] / ROWS + r.
template <int ROWS>
__device__ __forceinline__ int first_group(const AdjustParams& p, int r) {
  return min(max(__ldg(p.row_off + r), 0), p.rows) / ROWS + r;
}

constexpr int kWarps = kThreads / 32;
constexpr int kRowTokens = 512;   // of a request's rows in a stretch; more are looked up again for each row
constexpr int kPath = 64;         // a row's own tokens in a warp's part of a stretch; more 32 at a time

// kDeep: 16-byte pieces of a row that a lane has at a time.
template <typename T, int C, int kDeep>
struct Stretch {
  static constexpr int V = Piece<T>::V, kPart = 32 * kDeep * V, kParts = C / kPart, kWords = C / 32 + 2;
  static_assert(C % kPart == 0 && C / 32 <= kThreads - 2 && kPart <= 1024 && kPath >= 32);
  uint4 buffer[kWarps][32 * kDeep];                        // a part of a row, a warp's
  uint32_t count[C + V];                                   // times generated; the top bit: in the prompt
  uint32_t bias[C + V];                                    // 1 + place in the list of biases
  uint32_t some[kWords];                                   // tokens that occurred or have a bias
  uint32_t path[kWarps][kPart / 32];                       // tokens that the warp's row has in its path
  int row[kRowTokens];                                     // rows' own tokens in the stretch: row, token
  int rows, sum[kWarps];
  uint16_t token[kRowTokens];
  uint16_t before[kWords];                                 // set bits before a word
  uint16_t list[C + V];                                    // the set bits, ascending
  uint16_t entry[kWarps][kPath];
};

// How often the token at place `mine` of a part is in row i's path, a lane to a place: of the
// `of` listed rows' tokens, or of all rows' (tok).  Places [0, part) of the part begin at token
// t0 and place a0 of the stretch.  Warp-collective.  (Rare, and a function of its own: inlined,
// it cost the tree of 257 fp32 nodes 60 us against 56.)
__device__ __noinline__ uint32_t times_in_path(const int* row, const uint16_t* token, const int32_t* tok, int of, int t0,
                                               int a0, int part, const uint32_t* mask, int words, int i, int mine, int lane) {
  uint32_t times = 0;
  for (int e0 = 0; e0 < of; e0 += 32) {
    const int e = e0 + lane;
    int a = -1;
    if (e < of) {
      const int j = tok ? e : row[e];
      a = tok ? static_cast<int>(static_cast<unsigned>(__ldg(tok + e)) - static_cast<unsigned>(t0)) : token[e] - a0;
      const bool on = mask ? (j >> 5) < words && ((__ldg(mask + (j >> 5)) >> (j & 31)) & 1u) : j <= i;
      if (a < 0 || a >= part || !on) a = -1;
    }
    for (uint32_t who = __ballot_sync(0xffffffffu, a >= 0); who; who &= who - 1)
      times += __shfl_sync(0xffffffffu, a, __ffs(who) - 1) == mine;
  }
  return times;
}

template <typename T, int C, int kDeep, int ROWS>
__global__ void __launch_bounds__(kThreads, kDeep > 4 ? 3 : 4) logits_adjust_kernel(const AdjustParams p) {
  // Pieces lie on 16-byte boundaries, so a row's first one may begin up to V - 1 tokens
  // before it; stretch y is pieces y C / V .. of every row, tokens y C - V + 1 .. at most.
  using S = Stretch<T, C, kDeep>;
  constexpr int V = S::V, kPart = S::kPart, kParts = S::kParts;
  extern __shared__ __align__(16) uint8_t smem[];
  S& s = *reinterpret_cast<S*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, base = blockIdx.y * C - V;
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
  const int len = p.history ? min(max(__ldg(p.history_len + req), 0), p.history_ld) : 0;
  const int prompt = p.prompt_len ? __ldg(p.prompt_len + req) : 0;
  const bool track = rho != 1.f || phi != 0.f || pi != 0.f;
  const bool change = track || p.n_bias > 0;

  // a token's place in the stretch, if it has one
  // (a token that is none may have one too, before the row's first or behind its last: it
  // changes what is not written)
  auto from = [&](int t) { return static_cast<unsigned>(t) - static_cast<unsigned>(base); };
  auto place = [&](int t) { return from(t) < C + V ? static_cast<int>(from(t)) : -1; };
  auto note = [&](int a) { atomicOr(&s.some[a >> 5], 1u << (a & 31)); };
  const int words = p.mask ? min(p.mask_ld, (n + 31) / 32) : 0;
  auto sees = [&](int i, int j) {                          // whether row i's path holds row j (of the request)
    if (!p.mask) return j <= i;
    return (j >> 5) < words && ((__ldg(p.mask + (size_t)(row0 + i) * p.mask_ld + (j >> 5)) >> (j & 31)) & 1u);
  };

  if (change) {
    for (int a = tid; a < (C + V) / 4; a += kThreads) {
      reinterpret_cast<uint4*>(s.count)[a] = make_uint4(0, 0, 0, 0);
      if (p.n_bias > 0) reinterpret_cast<uint4*>(s.bias)[a] = make_uint4(0, 0, 0, 0);
    }
    if (tid < S::kWords) s.some[tid] = 0;
    for (int a = tid; a < kWarps * (kPart / 32); a += kThreads) (&s.path[0][0])[a] = 0;
    if (tid == 0) s.rows = 0;
    __syncthreads();
    if (track) {
      auto count = [&](int i, int t) {
        const int a = place(t);
        if (a < 0) return;
        i < prompt ? atomicOr(&s.count[a], 0x80000000u) : atomicAdd(&s.count[a], 1u);
        note(a);
      };
      // (four at a time, from the 16-byte boundary before the first)
      const int32_t* h = p.history + (size_t)req * p.history_ld;
      const int off = static_cast<int>(reinterpret_cast<uintptr_t>(h) >> 2) & 3;
      constexpr int kAtOnce = 8;
      for (int i = tid * 4 - off; i < len; i += kAtOnce * kThreads * 4) {
        int4 t[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int at = i + k * kThreads * 4;
          if (at >= len) continue;
          if (at >= 0 && at + 4 <= len) {
            t[k] = __ldg(reinterpret_cast<const int4*>(h + at));
          } else {
            auto one = [&](int e) { return at + e >= 0 && at + e < len ? __ldg(h + at + e) : -1; };
            t[k] = make_int4(one(0), one(1), one(2), one(3));
          }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int at = i + k * kThreads * 4;
          if (at >= len) break;
          // (most have none in the stretch)
          if (min(min(from(t[k].x), from(t[k].y)), min(from(t[k].z), from(t[k].w))) >= C + V) continue;
          count(at, t[k].x);
          count(at + 1, t[k].y);
          count(at + 2, t[k].z);
          count(at + 3, t[k].w);
        }
      }
      // The rows' own tokens: of a chain the ones before this group are everyone's past,
      // and the ones after it nobody's.
      if (p.tok)
        for (int j = tid; j < (p.mask ? n : i1); j += kThreads) {
          const int a = place(__ldg(p.tok + row0 + j));
          if (a < 0) continue;
          if (!p.mask && j < i0) {
            atomicAdd(&s.count[a], 1u);
            note(a);
          } else {
            const int e = atomicAdd(&s.rows, 1);
            if (e < kRowTokens) {
              s.row[e] = j;
              s.token[e] = static_cast<uint16_t>(a);
            }
          }
        }
    }
    for (int j = tid; j < p.n_bias; j += kThreads) {
      const int a = place(__ldg(p.bias_tok + (size_t)req * p.n_bias + j));
      if (a < 0) continue;
      atomicMax(&s.bias[a], static_cast<uint32_t>(j + 1));
      note(a);
    }
    __syncthreads();
    // the list: a thread to a word of bits, behind those of the words before
    uint32_t bits = tid < S::kWords ? s.some[tid] : 0u;
    int upto = __popc(bits);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) s.sum[warp] = upto;
    __syncthreads();
    int at = upto - __popc(bits);
    for (int w = 0; w < warp; ++w) at += s.sum[w];
    if (tid < S::kWords) s.before[tid] = static_cast<uint16_t>(at);
    for (; bits; bits &= bits - 1) s.list[at++] = static_cast<uint16_t>(tid * 32 + __ffs(bits) - 1);
    __syncthreads();
  }
  const int listed = change && track ? s.rows : 0;
  auto rank = [&](int a) { return s.before[a >> 5] + __popc(s.some[a >> 5] & ((1u << (a & 31)) - 1u)); };

  uint4* buffer = s.buffer[warp];
  T* value = reinterpret_cast<T*>(buffer);
  for (int item = warp; item < (i1 - i0) * kParts; item += kWarps) {
    const int i = i0 + item / kParts, part = item % kParts;
    const long long row = row0 + i;
    const T* in = static_cast<const T*>(p.logits) + row * p.ld;
    T* out = static_cast<T*>(p.out) + row * p.out_ld;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(in) / sizeof(T)) & (V - 1);
    const bool same = (static_cast<int>(reinterpret_cast<uintptr_t>(out) / sizeof(T)) & (V - 1)) == off;
    const int t0 = blockIdx.y * C + part * kPart - off;    // the part's first token
    uint4 u[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int t = t0 + (k * 32 + lane) * V;
      if (t >= p.vocab) continue;
      if (t >= 0 && t + V <= p.vocab) {
        u[k] = *reinterpret_cast<const uint4*>(in + t);
      } else {
        __align__(16) T e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = t + j >= 0 && t + j < p.vocab ? in[t + j] : T(0.f);
        u[k] = *reinterpret_cast<const uint4*>(e);
      }
    }
    uint32_t may[kDeep];                                   // a bit to an element
    const uint32_t* allowed = p.allowed ? p.allowed + row * p.allowed_ld : nullptr;
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int t = t0 + (k * 32 + lane) * V;
      may[k] = 0xFFFFFFFFu;
      if (!allowed || t >= p.vocab) continue;
      const int w = t >> 5, sh = t & 31;
      uint32_t x = w >= 0 ? __ldg(allowed + w) >> sh : 0u;
      if (sh + V > 32 && w < (p.vocab - 1) >> 5) x |= __ldg(allowed + w + 1) << (32 - sh);      // (sh > 0)
      may[k] = x;
    }
    if (change) {
      // places count from the part's first token from here on
      const int a0 = t0 - base, r0 = rank(a0), r1 = rank(a0 + kPart);
      // what the row's path has in this part
      // (from the list, or, if there are more, from all rows' tokens: only a tree has so many)
      int own = 0;
      const bool all = listed > kRowTokens;
      for (int e0 = 0, of = all ? n : listed; e0 < of; e0 += 32) {
        const int e = e0 + lane, j = all || e >= of ? e : s.row[e];
        const int a = e >= of ? -1 : (all ? static_cast<int>(from(__ldg(p.tok + row0 + e))) : s.token[e]) - a0;
        const bool on = a >= 0 && a < kPart && sees(i, j);
        const uint32_t who = __ballot_sync(0xffffffffu, on);
        const int at = own + __popc(who & ((1u << lane) - 1u));
        if (on) {
          atomicOr(&s.path[warp][a >> 5], 1u << (a & 31));
          if (at < kPath) s.entry[warp][at] = static_cast<uint16_t>(a);
        }
        own += __popc(who);
      }
      if (own > 0 || r1 > r0) {                            // (warp-uniform)
#pragma unroll
        for (int k = 0; k < kDeep; ++k) buffer[k * 32 + lane] = u[k];
        __syncwarp();
        auto fix = [&](int a, uint32_t more) {             // `more` times in the path
          const uint32_t b = p.n_bias > 0 ? s.bias[a0 + a] : 0u, count = s.count[a0 + a] + more;
          float y = to_f32(value[a]);
          if (b) y += __ldg(p.bias_val + (size_t)req * p.n_bias + b - 1);
          if (count) y = y > 0.f ? y / rho : y * rho;
          const uint32_t c = count & 0x7FFFFFFFu;
          if (c) y = y - phi * static_cast<float>(c) - pi;
          value[a] = from_f32<T>(y);
        };
        auto listed_ones = [&]() {                         // that are not in the path
          for (int e = r0 + lane; e < r1; e += 32) {
            const int a = s.list[e] - a0;
            if (!((s.path[warp][a >> 5] >> (a & 31)) & 1u)) fix(a, 0);
          }
        };
        if (own <= kPath) {
          listed_ones();
          for (int e = lane; e < own; e += 32) {
            const int a = s.entry[warp][e];
            uint32_t more = 0;
            bool first = true;
            for (int f = 0; f < own; ++f)
              if (s.entry[warp][f] == a) {
                first &= f >= e;
                ++more;
              }
            if (first) fix(a, more);
          }
        } else {
          // Too many to list: 32 of the path's different tokens at a time, ascending, one to a
          // lane, which counts it as all entries pass.  (A lane has a word of the path's bits.)
          listed_ones();
          uint32_t word = lane < kPart / 32 ? s.path[warp][lane] : 0u;
          int upto = __popc(word);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
          }
          const int distinct = __shfl_sync(0xffffffffu, upto, 31);
          int at = upto - __popc(word);
          for (int d0 = 0; d0 < distinct; d0 += 32) {
            __syncwarp();
            for (; word && at < d0 + 32; word &= word - 1)
              s.entry[warp][at++ - d0] = static_cast<uint16_t>(lane * 32 + __ffs(word) - 1);
            __syncwarp();
            const int mine = d0 + lane < distinct ? s.entry[warp][lane] : -1;
            const uint32_t more = times_in_path(s.row, s.token, all ? p.tok + row0 : nullptr, all ? n : listed, base + a0, a0,
                                                kPart, p.mask ? p.mask + (size_t)(row0 + i) * p.mask_ld : nullptr, words, i,
                                                mine, lane);
            if (mine >= 0) fix(mine, more);
          }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kDeep; ++k) u[k] = buffer[k * 32 + lane];
        if (own) {                                         // no path for the next row yet
          for (int w = lane; w < kPart / 32; w += 32) s.path[warp][w] = 0;
        }
        __syncwarp();
      }
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int t = t0 + (k * 32 + lane) * V;
      if (t >= p.vocab) continue;
      if ((may[k] & ((1u << V) - 1u)) != (1u << V) - 1u) {
        constexpr uint32_t kNone = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;     // -infinity
        uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t keep;
          if constexpr (sizeof(T) == 2) {                  // two bits, each to a half of the word
            const uint32_t two = may[k] >> (2 * j);
            keep = (two & 1u) * 0xFFFFu + (two & 2u) * 0x7FFF8000u;
          } else {
            keep = 0u - ((may[k] >> j) & 1u);
          }
          w[j] = (w[j] & keep) | (kNone & ~keep);
        }
        u[k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (t >= 0 && t + V <= p.vocab && same) {
        *reinterpret_cast<uint4*>(out + t) = u[k];
      } else {
        const T* e = reinterpret_cast<const T*>(&u[k]);
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (t + j >= 0 && t + j < p.vocab) out[t + j] = e[j];
      }
    }
  }
}

// Measured, us, 32 x 15 bf16 rows and a tree of 257 fp32 ones, of 151936 (at a time when they
// took 78 and 57): stretches of 4 KB, 2 KB of them to a warp at a time 78 and 62, 4 KB 89 and
// 62; of 8 KB 84 and 70 (the stretch of the commonest tokens is a longer one); groups of 32
// rows 77 and (4 KB to a warp) 57, of 8 rows 94 and 66.
template <typename T, int C, int kDeep, int ROWS>
void launch(const AdjustParams& p, cudaStream_t st) {
  using S = Stretch<T, C, kDeep>;
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(logits_adjust_kernel<T, C, kDeep, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(S));
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  const int groups = p.rows / ROWS + p.n_req;
  launch_k(logits_adjust_kernel<T, C, kDeep, ROWS>, dim3(groups, (p.vocab + S::V - 1 + C - 1) / C), dim3(kThreads), sizeof(S),
           st, p);
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
  DFL_REQUIRE(history == nullptr || history_ld <= kMaxHistory, "logits adjust: history rows longer than %d",
              kMaxHistory);
  DFL_REQUIRE(mask == nullptr || (mask_ld >= 1 && tok), "logits adjust: a mask needs words and tokens");
  DFL_REQUIRE(n_bias >= 0 && n_bias <= (1 << 20), "logits adjust: n_bias must be in [0, 2^20]");
  DFL_REQUIRE(allowed == nullptr || allowed_ld * 32 >= vocab, "logits adjust: allowed rows shorter than vocab");
  if (n_req == 0 || rows == 0) return DFLASH_OK;
  DFL_REQUIRE(logits && out && row_off, "logits adjust: null pointer argument");
  DFL_REQUIRE(n_bias == 0 || (bias_tok && bias_val), "logits adjust: null bias list");
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
    // A request's history is gone through for every stretch of each of its groups: requests of
    // one row, as in decoding, and many of a few rows take long stretches.  Otherwise few
    // CTAs' worth of rows take short ones.  Measured, us, rows of 151936 after 2048 tokens,
    // long / few / many, bf16 and fp32:
    //   256 x 1 83 / 261 / 140, 106 / 258 / 350;  16 x 1 7.3 / 17 / 10, 10 / 17 / 23;
    //   1 x 1 6.3 / 6.9 / 7.0, 6.4 / 6.3 / 7.4;   64 x 2 29 / 70 / 38, 42 / 74 / 93;
    //   32 x 4 23 / 38 / 22, 36 / 43 / 52;        1 x 4 12 / 7.3 / 7.3, 13 / 6.9 / 7.8;
    //   1 x 16 13 / 7.7 / 16, 14 / 7.4 / 11;      8 x 5 14 / 17 / 12, 15 / 19 / 15;
    //   32 x 8 46 / 73 / 36, 66 / 79 / 62;        1 x 257 45 / 67 / 33, 66 / 74 / 54.
    const bool few = (rows / 16 + n_req) * (long long)((vocab + 4095) / 4096) < 2 * num_sms();
    const bool apart = rows <= n_req || (!few && rows <= (dtype == DFLASH_BF16 ? 2ll : 4ll) * n_req);
    if (dtype == DFLASH_BF16)
      apart ? launch<__nv_bfloat16, 4096, 2, 4>(p, st)
            : few ? launch<__nv_bfloat16, 1024, 4, 4>(p, st) : launch<__nv_bfloat16, 2048, 4, 16>(p, st);
    else
      apart ? launch<float, 4096, 4, 4>(p, st) : few ? launch<float, 1024, 4, 4>(p, st) : launch<float, 1024, 8, 32>(p, st);
  }
  return check_launch("logits adjust");
}
