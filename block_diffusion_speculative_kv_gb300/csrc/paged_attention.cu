// Attention of new tokens over a paged KV cache.
//
// "Accelerating Speculative Decoding with Block Diffusion Draft Trees", section
// 3.4.5: a verification pass attends from every new token (one decoded token, a
// chain, a draft tree, a chunk of a prompt) to the request's cached context and
// to the new tokens it may see.  Per (row, head), with the running maximum m
// and sum l of a softmax over the visible keys in one pass:
//
//   s_t = q . k_t / sqrt(hd),  m' = max(m, s_t),
//   l' = l 2^(m - m') + 2^(s_t - m'),  o' = o 2^(m - m') + 2^(s_t - m') v_t
//
// (s in base-2 units), out = o / l.  m, l and o are fp32; the probabilities are
// rounded to bf16 for the second product, so that it runs on the tensor cores,
// and l sums them before that rounding.
//
// Work split.  A request's n tokens and the G query heads of a KV head are
// n * G query rows, TR to a tile.  All (request, KV head, tile) key ranges are
// laid end to end in steps of KS keys, and every CTA takes an equal share of
// that line, found on the device from row_off and pos0.  So ragged batches,
// single long contexts and prompt chunks all fill the SMs, and a tile that a
// share's border cuts is joined, in key order, by the last of its CTAs to
// arrive (a counter, no waiting).
//
// Rows whose mask hides a key must not meet that key's value: 0 * NaN is not 0.
// In steps where some row may not see some key, values that are not finite are
// looked for, and such a step takes its second product row by row.
#include <cmath>

#include <math_constants.h>

#include "kernels.h"
#include "mma_sync.cuh"
#include "paged_attention.h"

namespace dfl {

namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLazy = 8.f;   // a row's reference maximum may lag by this much (base-2 units)

// ---------------------------------------------------------------------------
// Few query rows (decoding): tiles of 16 rows on warp-level MMAs.
// ---------------------------------------------------------------------------
// Four warps; a step is 64 keys, 16 to each warp, which loads them for itself
// (cp.async, kStages deep) and keeps its own running softmax, so the main loop
// has no block barrier.  The four states meet when the tile ends.
constexpr int kRowsS = 16, kStepS = 64, kStagesS = 4, kThreadsS = 128;

template <int HD>
struct SmallSmem {
  static constexpr int kTile = 16 * HD * 2;                       // 16 keys of K or V
  static constexpr int kRing = 4 * kStagesS * 2 * kTile;
  static constexpr int kO = 4 * 16 * HD * 4;
  static constexpr int kBytes = kRing + kO + 4 * 16 * 8 + 16;
};

// Any element of a 16-byte chunk of bf16 that is infinite or NaN.
__device__ __forceinline__ bool not_finite8(const uint4& u) {
  auto bad = [](uint32_t w) {
    return (w & 0x7F800000u) == 0x7F800000u || (w & 0x00007F80u) == 0x00007F80u;
  };
  return bad(u.x) || bad(u.y) || bad(u.z) || bad(u.w);
}

template <int HD>
__global__ void __launch_bounds__(kThreadsS, 1) paged_attn_small_kernel(const PagedAttnParams p) {
  using S = SmallSmem<HD>;
  constexpr int kCh = HD / 8;                 // 16-byte chunks per key
  constexpr int kNt = HD / 8;                 // output column tiles of 8
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* ring = smem + warp * (kStagesS * 2 * S::kTile);
  float* sO = reinterpret_cast<float*>(smem + S::kRing);               // [4][16][HD]
  float2* sMl = reinterpret_cast<float2*>(smem + S::kRing + S::kO);    // [4][16]
  int* sLast = reinterpret_cast<int*>(sMl + 64);

  pdl_wait();
  pdl_trigger();
  const int grid = gridDim.x;
  const long long total = paged_total(p, kRowsS, kStepS, lane);
  const long long begin = paged_share(total, blockIdx.x, grid);
  const long long end = paged_share(total, blockIdx.x + 1, grid);
  if (begin >= end) return;
  PagedCursor c;
  paged_seek(p, kRowsS, kStepS, lane, begin, &c);
  c.left = end - begin;

  const __nv_bfloat16* pool_k = static_cast<const __nv_bfloat16*>(p.pv.k);
  const __nv_bfloat16* pool_v = static_cast<const __nv_bfloat16*>(p.pv.v);
  const int ra = lane >> 2, cq = (lane & 3) * 2;    // fragment row (and + 8) and column pair

  while (c.left > 0) {
    const PagedReq rq = c.rq;
    const int nG = rq.n * p.G, rho0 = c.j * kRowsS;
    const int kend = rq.key_end(c.j, p.G, kRowsS);
    const int n = static_cast<int>(min((long long)(c.n_steps - c.step), c.left));
    const int k0 = c.step * kStepS + warp * 16;     // this warp's first key of the piece
    const int head0 = c.g * p.G;

    auto load = [&](int i) {
      const int t0 = k0 + i * kStepS;
      uint8_t* dst = ring + (i % kStagesS) * 2 * S::kTile;
      if (i < n) {
        const int page = t0 < kend ? page_of(p.pv, c.r, t0) : -1;
        if (page < 0 && t0 < kend && lane == 0) record_status(p.status, DFLASH_ERR_INVALID_ARG);
        const long long at = page < 0 ? 0 : pool_row(p.pv, page, c.g, t0) * HD;
        const uint32_t dk = mmas::smem_u32(dst), dv = dk + S::kTile;
#pragma unroll
        for (int u = 0; u < kCh / 2; ++u) {
          const int ch = lane + 32 * u, row = ch / kCh, col = ch % kCh;
          const bool ok = page >= 0 && t0 + row < kend;
          mmas::cp_async16(dk + mmas::swz<HD>(row, col), pool_k + at + (ok ? row * HD + col * 8 : 0), ok);
          mmas::cp_async16(dv + mmas::swz<HD>(row, col), pool_v + at + (ok ? row * HD + col * 8 : 0), ok);
        }
      }
      mmas::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStagesS - 1; ++i) load(i);

    // this lane's rows: their token, and the first slot past what they see
    int tok[2], lim[2];
    uint32_t qf[HD / 16][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rho = rho0 + ra + 8 * h;
      const bool live = rho < nG;
      tok[h] = live ? rho / p.G : 0;
      lim[h] = live ? min(rq.p0 + (rq.masked ? 0 : tok[h] + 1), kend) : 0;
      const __nv_bfloat16* row =
          p.q + (long long)(rq.row0 + tok[h]) * p.q_ld + (long long)(head0 + (live ? rho % p.G : 0)) * HD;
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[kk][2 * e + h] =
              live ? __ldg(reinterpret_cast<const uint32_t*>(row + kk * 16 + 8 * e + cq)) : 0u;
    }
    // keys below `plain` are seen by every row of the tile
    const int plain = min(rq.masked ? rq.p0 : rq.p0 + rho0 / p.G + 1, kend);

    float o[kNt][4] = {};
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
    for (int i = 0; i < n; ++i) {
      load(i + kStagesS - 1);
      mmas::cp_async_wait<kStagesS - 1>();
      __syncwarp();
      const int t0 = k0 + i * kStepS;
      const uint8_t* tile = ring + (i % kStagesS) * 2 * S::kTile;
      const uint32_t sK = mmas::smem_u32(tile), sV = sK + S::kTile;
      if (t0 < kend) {
        float s[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          uint32_t b0, b1, b2, b3;
          mmas::ldsm_x4(sK + mmas::swz<HD>(((lane >> 4) << 3) + (lane & 7), 2 * kk + ((lane >> 3) & 1)),
                        b0, b1, b2, b3);
          mmas::mma16816(s[0], qf[kk], b0, b1);
          mmas::mma16816(s[1], qf[kk], b2, b3);
        }
        const bool all = t0 + 16 <= plain;       // warp-uniform
        uint32_t seen = 0xFFu;                   // bit 4 nt + e of s[nt][e]
        if (!all) {
          seen = 0;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = t0 + nt * 8 + cq + (e & 1), h = e >> 1;
              bool see = t < lim[h];
              if (rq.masked && !see && t >= rq.p0 && t < kend && rho0 + ra + 8 * h < nG) {
                const int b = t - rq.p0;
                see = (b >> 5) < p.mask_ld &&
                      ((__ldg(p.mask + (size_t)(rq.row0 + tok[h]) * p.mask_ld + (b >> 5)) >> (b & 31)) & 1u);
              }
              if (see) seen |= 1u << (4 * nt + e);
              else s[nt][e] = -CUDART_INF_F;
            }
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] *= p.scale_log2;
        float mx[2];
        bool raise = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          raise |= mx[h] > m[h] + kLazy || (m[h] == -CUDART_INF_F && mx[h] > m[h]);
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float m2 = fmaxf(m[h], mx[h]);
            const float f = m2 == -CUDART_INF_F ? 1.f : ex2(m[h] - m2);
            m[h] = m2;
            l[h] *= f;
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
              o[nt][2 * h] *= f;
              o[nt][2 * h + 1] *= f;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float base = m[h] == -CUDART_INF_F ? 0.f : m[h];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              s[nt][2 * h + e] = ex2(s[nt][2 * h + e] - base);
              l[h] += s[nt][2 * h + e];
            }
        }
        bool odd = false;
        if (!all) {
          for (int u = 0; u < kCh / 2; ++u)
            odd |= not_finite8(*reinterpret_cast<const uint4*>(tile + S::kTile + (lane + 32 * u) * 16));
          odd = __any_sync(0xffffffffu, odd);
        }
        if (!odd) {
          const uint32_t pf[4] = {mmas::pack_bf16(s[0][0], s[0][1]), mmas::pack_bf16(s[0][2], s[0][3]),
                                  mmas::pack_bf16(s[1][0], s[1][1]), mmas::pack_bf16(s[1][2], s[1][3])};
#pragma unroll
          for (int nt = 0; nt < kNt; nt += 2) {
            uint32_t b0, b1, b2, b3;
            mmas::ldsm_x4_t(sV + mmas::swz<HD>((((lane >> 3) & 1) << 3) + (lane & 7), nt + (lane >> 4)),
                            b0, b1, b2, b3);
            mmas::mma16816(o[nt], pf, b0, b1);
            mmas::mma16816(o[nt + 1], pf, b2, b3);
          }
        } else {
          // a value that is not finite: each row adds the keys it sees, one by one
          for (int key = 0; key < 16; ++key) {
            const int nt = key >> 3, from = (lane & ~3) | ((key & 7) >> 1);
            float pr[2];
            bool see[2];
            const unsigned sb = __shfl_sync(0xffffffffu, seen, from);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = nt ? ((key & 1) ? s[1][2 * h + 1] : s[1][2 * h])
                                 : ((key & 1) ? s[0][2 * h + 1] : s[0][2 * h]);
              pr[h] = __bfloat162float(__float2bfloat16_rn(__shfl_sync(0xffffffffu, x, from)));
              see[h] = (sb >> (4 * nt + 2 * h + (key & 1))) & 1u;
            }
#pragma unroll
            for (int t = 0; t < kNt; ++t) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(
                  tile + S::kTile + mmas::swz<HD>(key, t) + cq * 2);
              const float v0 = __uint_as_float(w << 16), v1 = __uint_as_float(w & 0xFFFF0000u);
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (see[h]) {
                  o[t][2 * h] += pr[h] * v0;
                  o[t][2 * h + 1] += pr[h] * v1;
                }
            }
          }
        }
      }
      __syncwarp();   // the slot may be loaded again
    }

    // the four warps' states
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      float* dst = sO + (warp * 16 + ra + 8 * h) * HD + cq;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
        *reinterpret_cast<float2*>(dst + nt * 8) = make_float2(o[nt][2 * h], o[nt][2 * h + 1]);
      if ((lane & 3) == 0) sMl[warp * 16 + ra + 8 * h] = make_float2(m[h], l[h]);
    }
    __syncthreads();
    constexpr int kCols = HD / 8;                        // thread: one row, kCols columns
    const int row = tid >> 3, col0 = (tid & 7) * kCols;
    float M = -CUDART_INF_F, L = 0.f, acc[kCols] = {};
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sMl[w * 16 + row].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float2 ml = sMl[w * 16 + row];
      if (ml.y == 0.f) continue;                         // this warp saw nothing for the row
      const float f = ex2(ml.x - M);
      L += f * ml.y;
#pragma unroll
      for (int x = 0; x < kCols; ++x) acc[x] += f * sO[(w * 16 + row) * HD + col0 + x];
    }
    const int rho = rho0 + row;
    auto write = [&]() {
      if (rho >= nG) return;
      const float inv = 1.f / L;                         // a row that saw no key: zeros
      __nv_bfloat16* dst = p.out + (long long)(rq.row0 + rho / p.G) * p.out_ld +
                           (long long)(head0 + rho % p.G) * HD + col0;
#pragma unroll
      for (int x = 0; x < kCols; x += 8) {
        uint32_t w4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w4[e] = L == 0.f ? 0u : mmas::pack_bf16(acc[x + 2 * e] * inv, acc[x + 2 * e + 1] * inv);
        *reinterpret_cast<uint4*>(dst + x) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
      }
    };
    const long long at = end - c.left, unit0 = at - c.step;
    if (n == c.n_steps) {
      write();
    } else {
      const int c0 = paged_owner(total, unit0, grid);
      const int c1 = paged_owner(total, unit0 + c.n_steps - 1, grid);
      const size_t slot = (size_t)blockIdx.x * 2 + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0);
      float* po = p.part_o + (slot * kRowsS + row) * HD + col0;
#pragma unroll
      for (int x = 0; x < kCols; x += 4)
        *reinterpret_cast<float4*>(po + x) = make_float4(acc[x], acc[x + 1], acc[x + 2], acc[x + 3]);
      if ((tid & 7) == 0) p.part_ml[slot * kRowsS + row] = make_float2(M, L);
      __threadfence();
      __syncthreads();
      if (tid == 0) *sLast = atomicAdd(p.arrive + c0, 1) == c1 - c0;
      __syncthreads();
      if (*sLast) {
        __threadfence();
        if (tid == 0) p.arrive[c0] = 0;                  // for the next call
        M = -CUDART_INF_F;
        L = 0.f;
#pragma unroll
        for (int x = 0; x < kCols; ++x) acc[x] = 0.f;
        for (int cc = c0; cc <= c1; ++cc)
          M = fmaxf(M, __ldcg(p.part_ml + ((size_t)cc * 2 + (cc == c0)) * kRowsS + row).x);
        for (int cc = c0; cc <= c1; ++cc) {
          const size_t s2 = ((size_t)cc * 2 + (cc == c0)) * kRowsS + row;
          const float2 ml = __ldcg(p.part_ml + s2);
          if (ml.y == 0.f) continue;
          const float f = ex2(ml.x - M);
          L += f * ml.y;
#pragma unroll
          for (int x = 0; x < kCols; x += 4) {
            const float4 v4 = __ldcg(reinterpret_cast<const float4*>(p.part_o + s2 * HD + col0 + x));
            acc[x] += f * v4.x;
            acc[x + 1] += f * v4.y;
            acc[x + 2] += f * v4.z;
            acc[x + 3] += f * v4.w;
          }
        }
        write();
      }
    }
    c.left -= n;
    mmas::cp_async_wait<0>();
    __syncthreads();                                     // sO and the ring are free again
    if (c.left > 0) paged_next(p, kRowsS, kStepS, &c);
  }
}

template <int HD>
void launch_small(const PagedAttnParams& p, int grid, cudaStream_t st) {
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(paged_attn_small_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         SmallSmem<HD>::kBytes);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  TraceScope ts("paged_attn_small", st);
  launch_k(paged_attn_small_kernel<HD>, dim3(grid), dim3(kThreadsS), SmallSmem<HD>::kBytes, st, p);
}

constexpr int kMaxTileRows = 16;

// Header, arrival counters, (max, sum) pairs, partial rows.
struct PagedWs {
  size_t arrive, ml, o, bytes;
};
PagedWs paged_ws(int grid, int head_dim) {
  PagedWs w;
  w.arrive = 256;
  w.ml = w.arrive + align_up((size_t)grid * sizeof(int), 256);
  w.o = w.ml + align_up((size_t)grid * 2 * kMaxTileRows * sizeof(float2), 256);
  w.bytes = w.o + (size_t)grid * 2 * kMaxTileRows * head_dim * sizeof(float);
  return w;
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

size_t dflash_paged_attention_workspace_bytes(int n_q, int n_kv, int head_dim) {
  if (n_kv < 1 || n_q < n_kv || n_q % n_kv || (head_dim != 64 && head_dim != 128)) return 0;
  return paged_ws(num_sms(), head_dim).bytes;
}

dflash_status dflash_paged_attention(const dflash_pages* pages, int n_req, int n_rows, int n_q,
                                     const int32_t* row_off, const int32_t* pos0, int max_rows,
                                     const void* q, long long q_ld, const uint32_t* mask,
                                     int mask_ld, void* out, long long out_ld, void* ws,
                                     size_t ws_bytes, void* stream) {
  PagedAttnParams p{};
  const dflash_status s = check_pages(pages, "paged attention", &p.pv);
  if (s) return s;
  const int hd = pages->head_dim;
  if (pages->dtype != DFLASH_BF16)
    return set_error(DFLASH_ERR_UNSUPPORTED, "paged attention: the cache must be bf16");
  DFL_REQUIRE(n_req >= 0 && n_rows >= 0 && max_rows >= 0, "paged attention: sizes must be >= 0");
  DFL_REQUIRE(n_q >= pages->n_kv && n_q % pages->n_kv == 0,
              "paged attention: n_q must be a multiple of n_kv");
  DFL_REQUIRE((long long)n_rows * n_q < (1ll << 31), "paged attention: rows x heads exceed 2^31");
  DFL_REQUIRE(q_ld >= (long long)n_q * hd && out_ld >= (long long)n_q * hd && q_ld % 8 == 0 &&
                  out_ld % 8 == 0,
              "paged attention: row strides too small or not multiples of 8");
  DFL_REQUIRE(mask == nullptr || (mask_ld >= 1 && (long long)mask_ld * 32 >= max_rows),
              "paged attention: mask rows shorter than max_rows");
  if (n_req == 0 || n_rows == 0) return DFLASH_OK;
  DFL_REQUIRE(row_off && pos0 && q && out, "paged attention: null pointer argument");
  DFL_REQUIRE(((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) == 0,
              "paged attention: q and out must be 16-byte aligned");
  const int grid = num_sms();
  const PagedWs w = paged_ws(grid, hd);
  if (!ws || ws_bytes < w.bytes)
    return set_error(DFLASH_ERR_WORKSPACE, "paged attention workspace needs %zu bytes, got %zu",
                     w.bytes, ws_bytes);
  DFL_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 15) == 0,
              "paged attention: the workspace must be 16-byte aligned");
  p.n_req = n_req;
  p.n_rows = n_rows;
  p.G = n_q / pages->n_kv;
  p.row_off = row_off;
  p.pos0 = pos0;
  p.mask = mask;
  p.mask_ld = mask_ld;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_ld = q_ld;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_ld = out_ld;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(hd));
  char* b = static_cast<char*>(ws);
  p.arrive = reinterpret_cast<int*>(b + w.arrive);
  p.part_ml = reinterpret_cast<float2*>(b + w.ml);
  p.part_o = reinterpret_cast<float*>(b + w.o);
  p.status = reinterpret_cast<int*>(b);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  hd == 128 ? launch_small<128>(p, grid, st) : launch_small<64>(p, grid, st);
  return check_launch("paged attention");
}

}  // extern "C"
