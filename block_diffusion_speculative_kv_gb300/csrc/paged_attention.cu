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
// single long contexts and prompt chunks all fill the SMs.  A tile that shares'
// borders cut is joined, in key order, by the last of its CTAs to arrive (a
// counter, no waiting), or, where tiles fall into many parts, by a second kernel.
//
// Rows whose mask hides a key must not meet that key's value: 0 * NaN is not 0.
// In steps where some row may not see some key, values that are not finite are
// looked for: they count as zeros in the second product, and rows that see one take
// the value itself.  So what no row sees changes no bit of a result.
#include <cmath>

#include <math_constants.h>

#include "gemm.h"
#include "kernels.h"
#include "mma_sync.cuh"
#include "paged_attention.h"
#include "ptx.cuh"

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
// Two CTAs share an SM: one streams while the other begins or ends a tile.  Memory
// bounds it: 32 requests of one token over 512 .. 8192 slots (head size 128, 8 KV heads)
// take 99 us, 6.2 TB/s of the 6.8 that a copy reaches; with one CTA to an SM 136.  One
// request over 2048 slots takes 10 us: launch, plan, one step and the join.
constexpr int kRowsS = 16, kStepS = 64, kStagesS = 3, kThreadsS = 128, kPerSmS = 2;
// Parts of a tile whose loads are in flight when they are joined (8 / 16 / 20: one row over
// 2048 slots 10.0 / 9.9 / 9.6 us, four rows 15.6 / 15.5 / 14.1, one over 500 9.0 / 9.2 / 9.3).
constexpr int kJoinS = 20;
using GeoS = PagedGeo<kRowsS, kStepS, 4, kRowsS, 2>;

template <int HD>
struct SmallSmem {
  static constexpr int kTile = 16 * HD * 2;                       // 16 keys of K or V
  static constexpr int kRing = 4 * kStagesS * 2 * kTile;
  static constexpr int kBytes = kRing + 4 * 16 * 8 + 16;
  static constexpr int kLd = HD + 8;                              // of a state's rows: no bank conflicts
  static_assert(4 * 16 * kLd * 4 <= kRing, "the warps' states meet in the idle ring");
};

// Any element of a 16-byte chunk of bf16 that is infinite or NaN.
__device__ __forceinline__ bool not_finite8(const uint4& u) {
  auto bad = [](uint32_t w) {
    return (w & 0x7F800000u) == 0x7F800000u || (w & 0x00007F80u) == 0x00007F80u;
  };
  return bad(u.x) || bad(u.y) || bad(u.z) || bad(u.w);
}

__device__ __forceinline__ uint32_t zero_not_finite(uint32_t w) {
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  if ((w & 0x00007F80u) == 0x00007F80u) w &= 0xFFFF0000u;
  return w;
}

template <int HD>
__global__ void __launch_bounds__(kThreadsS, kPerSmS) paged_attn_small_kernel(const PagedAttnParams p) {
  using S = SmallSmem<HD>;
  constexpr int kCh = HD / 8;                 // 16-byte chunks per key
  constexpr int kNt = HD / 8;                 // output column tiles of 8
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* ring = smem + warp * (kStagesS * 2 * S::kTile);
  float* sO = reinterpret_cast<float*>(smem);                          // [4][16][kLd], in the ring
  float2* sMl = reinterpret_cast<float2*>(smem + S::kRing);            // [4][16]
  int* sLast = reinterpret_cast<int*>(sMl + 64);

  pdl_wait();
  pdl_trigger();
  long long total, end;                                  // the line, and the end of this CTA's share
  PagedCursor c;
  paged_plan<GeoS>(p, lane, &total, &end, &c);

  const __nv_bfloat16* pool_k = static_cast<const __nv_bfloat16*>(p.pv.k);
  const __nv_bfloat16* pool_v = static_cast<const __nv_bfloat16*>(p.pv.v);
  const int ra = lane >> 2, cq = (lane & 3) * 2;    // fragment row (and + 8) and column pair

  for (PagedPiece pc; c.left > 0; paged_next<GeoS>(p, pc, &c)) {
    pc = PagedPiece::of<GeoS>(c);
    if (pc.n <= 0) continue;
    const PagedReq rq = c.rq;
    const int nG = rq.n * p.heads.G, rho0 = c.j * kRowsS;
    const int kend = rq.key_end<GeoS>(c.j, p.heads);
    const int n = pc.n;
    const int k0 = pc.first * kStepS + warp * 16;   // this warp's first key of the piece
    const int head0 = c.g * p.heads.G;

    bool missing = false;                       // a page is not there (warp-uniform)
    auto load = [&](int i) {
      const int t0 = k0 + i * kStepS;
      uint8_t* dst = ring + (i % kStagesS) * 2 * S::kTile;
      if (i < n) {
        const int page = t0 < kend ? page_of(p.pv, c.r, t0) : -1;
        missing |= page < 0 && t0 < kend;
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
      tok[h] = live ? p.heads.quot(rho) : 0;
      lim[h] = live ? min(rq.p0 + (rq.masked ? 0 : tok[h] + 1), kend) : 0;
      const __nv_bfloat16* row =
          p.q + (long long)(rq.row0 + tok[h]) * p.q_ld + (long long)(head0 + (live ? rho - tok[h] * p.heads.G : 0)) * HD;
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[kk][2 * e + h] =
              live ? __ldg(reinterpret_cast<const uint32_t*>(row + kk * 16 + 8 * e + cq)) : 0u;
    }
    // keys below `plain` are seen by every row of the tile
    const int plain = min(rq.masked ? rq.p0 : rq.p0 + p.heads.quot(rho0) + 1, kend);

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
        if (odd) {
          // A value that is not finite: rows that see it take the value itself (times any
          // weight it is the same inf or NaN), and it counts as zero in the product.
          for (int key = 0; key < 16; ++key) {
            const int nt = key >> 3, from = (lane & ~3) | ((key & 7) >> 1);
            const unsigned sb = __shfl_sync(0xffffffffu, seen, from);
#pragma unroll
            for (int t = 0; t < kNt; ++t) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(
                  tile + S::kTile + mmas::swz<HD>(key, t) + cq * 2);
              const float v[2] = {__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (((sb >> (4 * nt + 2 * h + (key & 1))) & 1u) && !(fabsf(v[e]) <= CUDART_MAX_NORMAL_F))
                    o[t][2 * h + e] += v[e];
            }
          }
          __syncwarp();
          for (int u = 0; u < kCh / 2; ++u) {
            uint4* w = reinterpret_cast<uint4*>(ring + (i % kStagesS) * 2 * S::kTile + S::kTile) + lane + 32 * u;
            *w = make_uint4(zero_not_finite(w->x), zero_not_finite(w->y), zero_not_finite(w->z), zero_not_finite(w->w));
          }
          __syncwarp();
        }
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
      }
      __syncwarp();   // the slot may be loaded again
    }

    if (missing)
      for (int t0 = k0; t0 < min(k0 + n * kStepS, kend); t0 += kStepS)
        if (page_of(p.pv, c.r, t0) < 0 && paged_seen<GeoS>(p, c, t0, min(t0 + 16, kend), lane) && lane == 0)
          record_status(p.status, DFLASH_ERR_INVALID_ARG);
    if (warp == 0) paged_past<GeoS>(p, c, lane);

    // the four warps' states, of the tile's live rows
    const int live = min(kRowsS, nG - rho0);
    mmas::cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (ra + 8 * h >= live) continue;
      float* dst = sO + (warp * 16 + ra + 8 * h) * S::kLd + cq;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
        *reinterpret_cast<float2*>(dst + nt * 8) = make_float2(o[nt][2 * h], o[nt][2 * h + 1]);
      if ((lane & 3) == 0) sMl[warp * 16 + ra + 8 * h] = make_float2(m[h], l[h]);
    }
    __syncthreads();
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
    const bool whole = n == pc.all;
    int c0 = 0, c1 = 0;
    if (!whole) paged_owners<GeoS>(c, total, end - c.left - c.at, pc.all, &c0, &c1);
    const int bid = blockIdx.x;
    const size_t slot = (size_t)bid * 2 + (bid == c0 ? 1 : 0);
    for (int i = tid; i < items; i += kThreadsS) {
      const int row = i / (HD / 4), col = i % (HD / 4) * 4;
      float M = -CUDART_INF_F, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, sMl[w * 16 + row].x);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 ml = sMl[w * 16 + row];
        if (ml.y == 0.f) continue;                       // this warp saw nothing for the row
        const float f = ex2(ml.x - M);
        L += f * ml.y;
        add(acc, f, *reinterpret_cast<const float4*>(sO + (w * 16 + row) * S::kLd + col));
      }
      if (whole) {
        write(row, col, acc, L);
      } else {
        *reinterpret_cast<float4*>(p.part_o + (slot * kRowsS + row) * HD + col) = acc;
        if (col == 0) p.part_ml[slot * kRowsS + row] = make_float2(M, L);
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
        float2* sPart = reinterpret_cast<float2*>(smem);
        const int parts = c1 - c0 + 1;
        for (int i = tid; i < parts * kRowsS; i += kThreadsS) {
          const int cc = c0 + i / kRowsS;
          sPart[i] = i % kRowsS < live
                         ? __ldcg(p.part_ml + ((size_t)cc * 2 + (cc == c0)) * kRowsS + i % kRowsS)
                         : make_float2(-CUDART_INF_F, 0.f);
        }
        __syncthreads();
        for (int i = tid; i < items; i += kThreadsS) {
          const int row = i / (HD / 4), col = i % (HD / 4) * 4;
          float M = -CUDART_INF_F, L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; k < parts; ++k) M = fmaxf(M, sPart[k * kRowsS + row].x);
          for (int k0 = 0; k0 < parts; k0 += kJoinS) {    // their loads in flight
            float4 v[kJoinS];
#pragma unroll
            for (int k = 0; k < kJoinS; ++k) {
              const int cc = c0 + min(k0 + k, parts - 1);
              v[k] = __ldcg(reinterpret_cast<const float4*>(
                  p.part_o + (((size_t)cc * 2 + (cc == c0)) * kRowsS + row) * HD + col));
            }
#pragma unroll
            for (int k = 0; k < kJoinS; ++k) {
              const float2 ml = sPart[min(k0 + k, parts - 1) * kRowsS + row];
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
    __syncthreads();                                     // the ring is free again
  }
}

template <int HD>
void launch_small(const PagedAttnParams& p, cudaStream_t st) {
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(paged_attn_small_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         SmallSmem<HD>::kBytes);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  TraceScope ts("paged_attn_small", st);
  launch_k(paged_attn_small_kernel<HD>, dim3(num_sms() * kPerSmS), dim3(kThreadsS), SmallSmem<HD>::kBytes, st, p);
}

// ---------------------------------------------------------------------------
// Many query rows (chains, trees, prompt chunks): tensor-core tiles.
// ---------------------------------------------------------------------------
// A tile is NG MMA tiles of 128 query rows, against steps of 128 keys:
//   S_x = Q_x K_t^T   (x < NG; accumulators S_x in TMEM)
//   O_x += P_x V_t    (P_x in TMEM over S_x's columns, as the A operand; O_x in TMEM)
// NG = 2 (prompt chunks, trees): two softmax groups of four warps, one thread to
// a row, take turns with the tensor cores: while group 0 turns S_0 into P_0, the
// cores run P_1 V and the next S_1, and both MMA tiles share K and V.  A tile of
// at most 128 rows is given to both groups, which take every other key step each
// and join their halves at the end.  NG = 1 (chains): tiles of 64 rows, the first
// half of an MMA tile (the other half multiplies whatever follows Q in shared
// memory, and nobody reads it), with half an SM's shared memory and TMEM, so that
// two CTAs share an SM: memory bounds these tiles, and one CTA streams while the
// other begins or ends a tile.
// What bounds them.  NG = 1: memory; 32 requests of 16 rows over 512 .. 8192 slots take
// 110 us, 5.5 TB/s.  NG = 2: a prompt chunk of 2048 rows over 8192 slots takes 230 us,
// 1.35 PFLOP/s.  A step of a group is a chain: 420 clocks to read the scores from TMEM,
// 400 for their maximum, 1250 for the probabilities, 900 for the rest of P V and the
// next scores; the other group's hides behind it.  The tensor cores need 2830 a step at
// least, not the 2080 of their rate: both operands of the scores come from shared
// memory, 8 KB to an MMA of 64 clocks, which is all that it delivers.  The exponential
// unit is not it: with one exponential in four as a polynomial on the FMA pipe the chunk
// took 262 us against 237, with one in eight 241; nor did it help to read half the scores
// while the other half's maximum is found (240 against 231), or to form the first 32 keys
// of P before the maximum is known (231).  Small tiles, short
// contexts: beginning and ending a tile, about 6 us for the query rows on their way in
// and O on its way out, 257 rows over 8192 slots 56 us.
// After the softmax warps, one loads (TMA, a ring of K and V tiles that runs ahead
// over tile borders; a box is a page, or a slot of a larger one), the next one
// issues the MMAs.  A row's O is rescaled only when its maximum has risen by more
// than 8 (base-2 units) over the reference in use.  Every wait is bounded (2 s, or the limit in
// the workspace header); on expiry the CTA records DFLASH_ERR_TIMEOUT, lets its copies and
// MMAs land (2 s at most), frees TMEM and returns.
constexpr int kStepT = 128;
// Registers with NG = 2: the launch's 168 for each of three warpgroups, of which
// the softmax groups take 216 (a row of scores in registers) and the other one
// keeps 72: 2 * 216 + 72 = 3 * 168.
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * 168, "register split");
constexpr uint64_t kTimeoutNs = 2000000000ull, kMaxLimitNs = 60000000000ull;

struct PagedTcMaps {
  CUtensorMap k, v;    // pools as [n_pages * n_kv * page_size][HD], box 64 x min(page_size, slot)
};

template <int HD, int NG>
struct Tc {
  static constexpr int kGroup = NG == 2 ? 128 : 64;         // rows, and threads, of a softmax group
  static constexpr int kRows = kGroup * NG, kWarps = kRows / 32;
  static constexpr int kThreads = NG == 2 ? 384 : 128, kPerSm = NG == 2 ? 1 : 2;
  using Geo = PagedGeo<kRows, kStepT, NG == 2 ? 12 : 3, 128, NG == 2 ? 1 : 3>;
  static constexpr int kAtomQ = kGroup * 128;               // 64 columns of a group's rows of Q
  static constexpr int kTileQ = (HD / 64) * kAtomQ;
  static constexpr int kKeys = NG == 2 ? 128 : 64;          // of a ring slot
  static constexpr int kPer = kStepT / kKeys;               // slots of a step's K, or V
  // Keys of P that go out first: what the tensor cores do with the rest before the
  // next scores lies on the chain (64 / 96 keys first: the chunk above 237 / 231 us).
  // NG = 1: a slot of V.
  static constexpr int kEarly = NG == 2 ? 96 : 64;
  static constexpr int kAtom = kKeys * 128, kSlot = (HD / 64) * kAtom;
  static constexpr int kSlots = HD == 64 ? 8 : NG == 2 ? 5 : 6;
  static constexpr int kRing = NG * kTileQ;                 // after Q
  static constexpr int kBar = kRing + kSlots * kSlot;
  static constexpr int kBytes = kBar + (NG == 2 ? 2048 : 1024);
  static constexpr int kTmem = 256 * NG;                    // S_x at 128 x (P_x over it), then O_x
  static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "shared memory of an SM");
};

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

// Whether a value among eight is infinite or NaN: x * 0 is NaN for those, and
// sticks in the sum.
__device__ __forceinline__ void gather_bad(__nv_bfloat162& acc, const uint4& u) {
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int e = 0; e < 4; ++e) acc = __hfma2(h[e], zero, acc);
}

template <int HD, int NG>
__global__ void __launch_bounds__(Tc<HD, NG>::kThreads, Tc<HD, NG>::kPerSm)
paged_attn_tc_kernel(const __grid_constant__ PagedTcMaps maps, const PagedAttnParams p) {
  using S = Tc<HD, NG>;
  using Geo = typename S::Geo;
  constexpr int R = S::kSlots, kPer = S::kPer;
  extern __shared__ __align__(1024) uint8_t smem_tc[];
  uint8_t* smem = smem_tc;
  if (ptx::smem_addr(smem) & 1023) {                         // (the swizzle counts on it)
    record_status(p.status, DFLASH_ERR_UNSUPPORTED);
    return;
  }
  uint8_t* sQ = smem;                                        // [NG][HD / 64][128][64] bf16
  uint8_t* sKV = smem + S::kRing;                            // slots of [HD / 64][kKeys][64]
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint64_t* full = bar;                                      // [R] tile landed
  uint64_t* empty = bar + R;                                 // [R] tile read
  uint64_t* q_full = bar + 2 * R;
  uint64_t* s_ready = q_full + 1;                            // [NG]
  uint64_t* p_ready = q_full + 3;                            // [NG][half]
  uint64_t* pv_done = q_full + 7;                            // [NG]
  uint64_t* drain = q_full + 9;
  uint64_t* wait_ns = q_full + 10 + (threadIdx.x >> 5);      // limit of a wait, a word to a warp
  uint32_t* tslot = reinterpret_cast<uint32_t*>(q_full + 22);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  volatile int* s_last = reinterpret_cast<volatile int*>(tslot + 2);    // [2]
  // keys with a value that is not finite: [group][step % 4][word].  Group 1 may
  // still read group 0's of step t when group 0 is at step t + 2, not later.
  volatile uint32_t* odd_keys = tslot + 4;
  float2* sMl = reinterpret_cast<float2*>(tslot + 36);       // [128] (NG = 2)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < R; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    ptx::mbar_init(q_full, S::kWarps);
    for (int x = 0; x < NG; ++x) {
      ptx::mbar_init(&s_ready[x], 1);
      ptx::mbar_init(&p_ready[2 * x], S::kGroup / 32);
      ptx::mbar_init(&p_ready[2 * x + 1], S::kGroup / 32);
      ptx::mbar_init(&pv_done[x], 1);
    }
    ptx::mbar_init(drain, 1);
    *abort = 0;
    ptx::fence_mbar_init();
  }
  constexpr int kLoad = S::kWarps, kIssue = S::kWarps + 1;    // warps
  constexpr int GT = S::kGroup;
  if (warp == kIssue) {
    ptx::tmem_alloc(tslot, S::kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tbase = *tslot;
  const uint32_t tbase_o = tbase + 128 * NG;                 // O_x at 128 x from here

  pdl_wait();
  pdl_trigger();
  long long total, end;
  PagedCursor c;
  // the workspace header's limit (dflash_workspace_set_wait_limit), read beside the plan
  const uint64_t limit = *reinterpret_cast<const volatile uint64_t*>(p.status + 2);
  paged_plan<Geo>(p, lane, &total, &end, &c);
  if (lane == 0) *wait_ns = limit == 0 || limit > kMaxLimitNs ? kTimeoutNs : limit;
  __syncwarp();

  auto fail = [&]() {
    if (!*abort) record_status(p.status, DFLASH_ERR_TIMEOUT);
    *abort = 1;
  };
  // bounded waits; the loader and the issuer back off between polls, since they
  // share schedulers with the softmax
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (ptx::mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!ptx::mbar_try_wait(b, parity))
      if (*abort || global_ns() - t0 > *wait_ns) return false;
    return true;
  };

  if (warp >= kLoad) {
  if constexpr (NG == 2) ptx::regs_dec<kRegsOther>();
  if (warp == kLoad) {
    // ---------------- loads ----------------
    const int box = min(1 << p.pv.page_shift, S::kKeys);
    const int nb = kStepT / box;                             // boxes of a step's K, or V
    const int per_slot = S::kKeys / box;
    const uint64_t pol = ptx::policy_evict_last();
    if (lane == 0) {
      ptx::prefetch_tmap(&maps.k);
      ptx::prefetch_tmap(&maps.v);
    }
    const int nowhere = (p.pv.n_pages * p.pv.n_kv) << p.pv.page_shift;   // past the pool: zeros
    uint32_t it = 0;                                         // tiles loaded
    bool ok = true;
    for (PagedPiece pc; c.left > 0 && ok; paged_next<Geo>(p, pc, &c)) {
      pc = PagedPiece::of<Geo>(c);
      if (pc.n <= 0) continue;
      const int n = pc.n, kend = c.rq.key_end<Geo>(c.j, p.heads);
      const int32_t* table = p.pv.table + (size_t)c.r * p.pv.table_ld;
      // this lane's box of step i: its first slot, and its page's table entry
      // (asked for one step ahead; kend lies within the table)
      auto slot_of = [&](int i) { return (pc.first + i) * kStepT + lane * box; };
      auto entry_of = [&](int i) {
        const int t = slot_of(i);
        return lane < nb && i < n && t < kend ? __ldg(table + (t >> p.pv.page_shift)) : -1;
      };
      int entry = entry_of(0);
      bool missing = false;
      for (int i = 0; i < n && ok; ++i) {
        const int t = slot_of(i), page = entry;
        entry = entry_of(i + 1);
        const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.pv.n_pages);
        missing |= !there && lane < nb && t < kend;
        const int y = there ? static_cast<int>(pool_row(p.pv, page, c.g, t)) : nowhere;
        for (int kv = 0; kv < 2 * kPer && ok; ++kv, ++it) {   // K's slots, then V's
          const int s = it % R, part = kv % kPer;
          ok = wait(&empty[s], (it / R & 1u) ^ 1u);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) ptx::mbar_arrive_expect_tx(&full[s], S::kSlot);
          __syncwarp();
          const int b = lane - part * per_slot;              // this lane's box in the slot
          if (b >= 0 && b < per_slot)
            for (int h = 0; h < HD / 64; ++h)
              ptx::tma_load_2d(sKV + s * S::kSlot + h * S::kAtom + b * box * 128,
                               kv >= kPer ? &maps.v : &maps.k, &full[s], 64 * h, y, pol);
        }
      }
      // pages that are not there: an error if some row of the tile sees their slots
      if (__any_sync(0xffffffffu, missing))
        for (int t0 = pc.first * kStepT; t0 < min((pc.first + n) * kStepT, kend); t0 += box)
          if (page_of(p.pv, c.r, t0) < 0 && paged_seen<Geo>(p, c, t0, min(t0 + box, kend), lane) && lane == 0)
            record_status(p.status, DFLASH_ERR_INVALID_ARG);
    }
    if (!ok && lane == 0) fail();
    // every copy must land before the CTA exits
    for (uint32_t s = 0; s < R; ++s) {
      if (it <= s) break;
      const uint32_t last = (it - 1 - s) / R;                // uses of slot s - 1
      ptx::mbar_wait_bounded(&full[s], last & 1u, kTimeoutNs, nullptr);
    }
  } else if (warp == kIssue) {
    // ---------------- MMA issue ----------------
    // The whole warp runs the loop, so that addresses and descriptors stay in
    // uniform registers; one elected lane issues.  Descriptors differ by their
    // address field alone: a constant is added to the tile's.
    const bool elected = ptx::elect_one();
    const uint64_t dq = ptx::sw128_kmajor_desc(ptx::smem_addr(sQ));
    const uint64_t dk = ptx::sw128_kmajor_desc(ptx::smem_addr(sKV));
    const uint64_t dv = ptx::sw128_mnmajor_desc(ptx::smem_addr(sKV), S::kAtom, 1024);
    constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(128, S::kKeys);
    constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(128, HD) | (1u << 16);   // B transposed
    uint32_t it = 0, unit = 0, np[2] = {0, 0};               // ring base, units, PV products of x
    uint32_t ks[kPer] = {}, vs[kPer] = {};                   // ring slots in use
    bool ok = true;
    for (PagedPiece pc; c.left > 0 && ok; paged_next<Geo>(p, pc, &c)) {
      pc = PagedPiece::of<Geo>(c);
      if (pc.n <= 0) continue;
      const int n = pc.n, nt = NG == 2 && min(c.rq.n * p.heads.G - c.j * S::kRows, S::kRows) > 128 ? 2 : 1;
      auto all = [&](bool landed) { return __all_sync(0xffffffffu, landed); };
      ok = all(wait(q_full, unit & 1u));
      const int jobs0 = NG == 1 || nt == 2 ? n : (n + 1) / 2, jobs1 = NG == 1 ? 0 : (nt == 2 ? n : n / 2);
      // group x's i-th job is this step; ring slots of a step: K's, V's
      auto step_of = [&](int x, int i) { return NG == 1 || nt == 2 ? i : 2 * i + x; };
      auto slot_at = [&](uint32_t at) { return __shfl_sync(0xffffffffu, at % R, 0); };
      // Waits that the loads decide come before the one that the softmax decides, and
      // between that one and the next scores there is nothing but MMAs.
      auto landed = [&](uint32_t at) { return all(wait(&full[at % R], at / R & 1u)); };
      auto scores = [&](int x, int i) {                      // one lane: S_x of job i
        const uint64_t q0 = dq + (nt == 2 ? x * (S::kTileQ >> 4) : 0);
#pragma unroll
        for (int part = 0; part < kPer; ++part) {
          const uint32_t s = ks[part];
          const uint64_t k0 = dk + s * (S::kSlot >> 4);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            ptx::mma_bf16(tbase + 128 * x + part * S::kKeys,
                          q0 + (((kk >> 2) * S::kAtomQ + (kk & 3) * 32) >> 4),
                          k0 + (((kk >> 2) * S::kAtom + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
          if (part == kPer - 1) ptx::mma_commit(&s_ready[x]);
          if (nt == 1 || x == 1) ptx::mma_commit(&empty[s]);
        }
      };
      auto wait_k = [&](int x, int i) {
        const uint32_t at = it + 2 * kPer * step_of(x, i);
        bool got = true;
#pragma unroll
        for (int part = 0; part < kPer; ++part) {
          ks[part] = slot_at(at + part);
          got = got && landed(at + part);
        }
        return got;
      };
      // job i of group x: P V, then the scores of job i + 1
      auto turn = [&](int x, int i, bool more) {
        const bool shared = nt == 2 && x == 1;               // group 0 has waited for these
        const uint32_t at = it + 2 * kPer * step_of(x, i) + kPer;
        if (!shared) {
#pragma unroll
          for (int part = 0; part < kPer; ++part) {
            vs[part] = slot_at(at + part);
            if (!landed(at + part)) return false;
          }
          if (more && !wait_k(x, i + 1)) return false;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {                        // P arrives in two halves
          if (!all(wait(&p_ready[2 * x + h], np[x] & 1u))) return false;
          ptx::tc_fence_after();
          if (elected) {
            const uint32_t s = vs[kPer == 2 ? h : 0];
            const uint64_t v0 = dv + s * (S::kSlot >> 4);
#pragma unroll
            for (int j = h * (S::kEarly / 16); j < (h ? kStepT : S::kEarly) / 16; ++j)
              ptx::mma_bf16_ta(tbase_o + 128 * x, tbase + 128 * x + j * 8,
                               v0 + (j % (S::kKeys / 16)) * (2048 >> 4), idesc_pv, (i > 0 || j > 0) ? 1u : 0u);
            if (h == 1) ptx::mma_commit(&pv_done[x]);
            if ((kPer == 2 || h == 1) && (nt == 1 || x == 1)) ptx::mma_commit(&empty[s]);
            if (h == 1 && more) scores(x, i + 1);
          }
          __syncwarp();
        }
        ++np[x];
        return true;
      };
      for (int x = 0; x < 2 && ok; ++x) {
        if (x == 1 && jobs1 == 0) break;
        if (nt == 1 || x == 0) ok = wait_k(x, 0);
        ptx::tc_fence_after();
        if (ok && elected) scores(x, 0);
        __syncwarp();
      }
      for (int i = 0; i < jobs0 && ok; ++i) {
        ok = turn(0, i, i + 1 < jobs0);
        if (ok && i < jobs1) ok = turn(1, i, i + 1 < jobs1);
      }
      it += 2 * kPer * n;
      ++unit;
      paged_past<Geo>(p, c, lane);
    }
    if (!ok && lane == 0) fail();
    // the MMAs already issued finish before TMEM is released
    if (unit > 0 || !ok) {
      if (elected) ptx::mma_commit(drain);
      __syncwarp();
      ptx::mbar_wait_bounded(drain, 0u, kTimeoutNs, nullptr);
    }
    __syncwarp();
  }
  } else {
    if constexpr (NG == 2) ptx::regs_inc<kRegsSoftmax>();
    // ---------------- softmax: group x = warp / 4, a row to a thread ----------------
    const int x = warp / (GT / 32), wg = warp % (GT / 32), row = wg * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wg * 32) << 16;
    const uint32_t aS = tbase + 128 * x + lane_off, aO = tbase_o + 128 * x + lane_off;
    const float sc = p.scale_log2;
    uint32_t it = 0, nj = 0;                                 // ring base, jobs of this group
    bool ok = true;
    if (p.cut && tid == 0) p.cut[blockIdx.x].c1 = -1;
    for (PagedPiece pc; c.left > 0; paged_next<Geo>(p, pc, &c)) {
      pc = PagedPiece::of<Geo>(c);
      if (pc.n <= 0) continue;
      const PagedReq rq = c.rq;
      const int n = pc.n, nG = rq.n * p.heads.G, tile0 = c.j * S::kRows;
      const int nt = NG == 2 && min(nG - tile0, S::kRows) > 128 ? 2 : 1;
      const int kend = rq.key_end<Geo>(c.j, p.heads);
      const int rho0 = tile0 + (nt == 2 ? x * GT : 0);       // first row of this group's MMA tile
      const int rho = rho0 + row;
      const bool live = rho < nG;
      const int tok = live ? p.heads.quot(rho) : 0, head = c.g * p.heads.G + (live ? rho - tok * p.heads.G : 0);
      const int jobs = NG == 1 || nt == 2 ? n : (n + 1 - x) / 2;
      // Q into shared memory (rows of 128 bytes, 128-byte swizzle): HD / 8 lanes
      // read a row, whose address its own lane knows
      if (nt == 2 || x == 0) {
        const unsigned long long mine = reinterpret_cast<unsigned long long>(
            p.q + (long long)(rq.row0 + tok) * p.q_ld + (long long)head * HD);
        const unsigned on = __ballot_sync(0xffffffffu, live);
        constexpr int kLines = 256 / HD;                     // rows of a round
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += kLines) {
          const int rr = r0 + lane / (HD / 8), ch = lane % (HD / 8);
          const uint4* src = reinterpret_cast<const uint4*>(__shfl_sync(0xffffffffu, mine, rr)) + ch;
          const uint4 u = (on >> rr) & 1u ? __ldg(src) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(sQ + x * S::kTileQ + (ch >> 3) * S::kAtomQ + (wg * 32 + rr) * 128 +
                                    (((ch & 7) ^ (rr & 7)) << 4)) = u;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(q_full);

      // first slot past what the row sees (causal), the mask row, and the keys
      // that every row of the warp, and of the whole tile, sees
      const int lim = live ? (rq.masked ? kend : min(rq.p0 + tok + 1, kend)) : 0;
      const uint32_t* mrow = rq.masked ? p.mask + (size_t)(rq.row0 + tok) * p.mask_ld : nullptr;
      const int first = p.heads.quot(min(rho0 + wg * 32, nG - 1));
      const int plain_w = rho0 + wg * 32 >= nG ? 0 : min(rq.masked ? rq.p0 : rq.p0 + first + 1, kend);
      const int plain_t = min(rq.masked ? rq.p0 : rq.p0 + p.heads.quot(tile0) + 1, kend);
      const bool dead = rho0 + wg * 32 >= nG;        // no live row in this warp
      float m_ref = -CUDART_INF_F, l = 0.f;
      // A step's P V ran with zeros for values that are not finite.  Once it is done
      // (the next scores are, or pv_done), a row that sees such a key takes the value
      // itself: times any weight it is the same inf or NaN.
      int late = -1;                                         // first key of that step, or none
      volatile uint32_t* late_note = odd_keys;
      uint32_t late_seen[4];
      auto repair = [&]() {
        if (late < 0 || dead) return;
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          uint32_t keys = late_note[b];
          const uint32_t sees = b == 0 ? late_seen[0] : b == 1 ? late_seen[1] : b == 2 ? late_seen[2] : late_seen[3];
          while (keys) {                                     // warp-uniform
            const int j = __ffs(keys) - 1;
            keys &= keys - 1;
            const int key = late + 32 * b + j, page = page_of(p.pv, c.r, key);
            if (page < 0) continue;
            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.pv.v) + pool_row(p.pv, page, c.g, key) * HD;
            const bool see = (sees >> j) & 1u;
#pragma unroll 1
            for (int cb = 0; cb < HD / 16; ++cb) {
              float o[16];
              ptx::tmem_ld_32x16(aO + 16 * cb, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float val = __bfloat162float(v[16 * cb + e]);
                if (see && !(fabsf(val) <= CUDART_MAX_NORMAL_F)) o[e] += val;
              }
              ptx::tmem_st_32x16(aO + 16 * cb, o);
              ptx::tmem_wait_st();
            }
          }
        }
      };
      // (after a wait has run out the loop only keeps the group's barriers company)
      for (int i = 0; i < jobs; ++i, ++nj) {
        const int t = NG == 1 || nt == 2 ? i : 2 * i + x, key0 = (pc.first + t) * kStepT;
        volatile uint32_t* noted = odd_keys + 16 * (nt == 2 ? 0 : x) + 4 * (t & 3);
        if (ok) ok = __all_sync(0xffffffffu, wait(&s_ready[x], nj & 1u));
        const bool check = key0 + kStepT > plain_t && (nt == 1 || x == 0);   // group-uniform
        uint32_t seen[4];
        const bool early = !check && !dead;                  // P goes out in two halves
        if (ok && !dead) {
          ptx::tc_fence_after();
          if (late >= 0) repair();
          const bool cut = key0 + kStepT > plain_w;          // some key is hidden from some row
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            seen[b] = 0xFFFFFFFFu;
            if (cut) {
              const int k = key0 + 32 * b;
              seen[b] = low_bits(lim - k);
              if (rq.masked && seen[b]) seen[b] &= seen_word(mrow, p.mask_ld, k - rq.p0);
            }
          }
          uint32_t u[4][32];
#pragma unroll
          for (int b = 0; b < 4; ++b) ptx::tmem_ld_32x32(aS + 32 * b, u[b]);
          ptx::tmem_wait_ld();
          if (cut) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((seen[b] >> j) & 1u)) u[b][j] = 0xff800000u;
          }
          float mx8[8];                                      // eight chains: latency
#pragma unroll
          for (int j = 0; j < 8; ++j) mx8[j] = __uint_as_float(u[0][j]);
#pragma unroll
          for (int j = 4; j < 64; ++j)
            mx8[j & 7] = fmaxf(fmaxf(mx8[j & 7], __uint_as_float(u[j >> 4][2 * (j & 15)])),
                               __uint_as_float(u[j >> 4][2 * (j & 15) + 1]));
          const float top = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                  fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]))) * sc;
          const bool raise = top > m_ref + kLazy || (m_ref == -CUDART_INF_F && top > m_ref);
          if (__any_sync(0xffffffffu, raise)) {
            const float f = raise ? (m_ref == -CUDART_INF_F ? 0.f : ex2(m_ref - top)) : 1.f;
            if (raise) m_ref = top;
            l *= f;
            if (i > 0) {
              // the products so far must be in O before it is scaled
              ok = __all_sync(0xffffffffu, wait(&pv_done[x], (nj - 1) & 1u));
              if (ok) {
                ptx::tc_fence_after();
#pragma unroll 1
                for (int b = 0; b < HD / 16; ++b) {
                  float o[16];
                  ptx::tmem_ld_32x16(aO + 16 * b, o);
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] *= f;
                  ptx::tmem_st_32x16(aO + 16 * b, o);
                }
              }
            }
          }
          const float base = m_ref == -CUDART_INF_F ? 0.f : m_ref;
          const float2 sc2 = make_float2(sc, sc), nb2 = make_float2(-base, -base);
          float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            float pk[16];                                      // (two bf16 each)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 y = __ffma2_rn(
                  make_float2(__uint_as_float(u[b][2 * j]), __uint_as_float(u[b][2 * j + 1])), sc2, nb2);
              const float2 w = make_float2(ex2(y.x), ex2(y.y));
              rs[j & 1] = __fadd2_rn(rs[j & 1], w);
              pk[j] = __uint_as_float(mmas::pack_bf16(w.x, w.y));
            }
            ptx::tmem_st_32x16(aS + 16 * b, pk);
            if (b == S::kEarly / 32 - 1 && early) {
              // the first keys of P may meet V while the others are formed
              ptx::tmem_wait_st();
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0 && ok) ptx::mbar_arrive(&p_ready[2 * x]);
            }
          }
          l += (rs[0].x + rs[0].y) + (rs[1].x + rs[1].y);
          ptx::tmem_wait_st();
        }
        bool odd = false;
        if (check) {
          // Some row may not see some key of this step: the values of keys past
          // the tile's last one become zeros, and so do values that are not
          // finite (their keys are noted, see below).
          const uint32_t v_at = it + 2 * kPer * t + kPer;
          bool landed = true;
          for (int part = 0; part < kPer && ok && landed; ++part)
            landed = wait(&full[(v_at + part) % R], (v_at + part) / R & 1u);
          ok = __all_sync(0xffffffffu, ok && landed);
          if (ptx::named_bar_or(1 + x, GT, !ok)) ok = false;
#pragma unroll
          for (int k0 = 0; k0 < kStepT; k0 += GT) {
            // this thread: one key, whose 16-byte chunks it takes in another order
            // than its neighbours (no bank conflicts)
            const int key = k0 + row;
            bool mine = false;
            if (ok) {
              const uint32_t s = (v_at + key / S::kKeys) % R;
              uint8_t* v = sKV + s * S::kSlot + (key % S::kKeys) * 128;
              auto chunk = [&](int ch) {
                return reinterpret_cast<uint4*>(v + (ch >> 3) * S::kAtom + (((ch & 7) ^ (row & 7)) << 4));
              };
              if (key0 + key >= kend) {
#pragma unroll
                for (int ch = 0; ch < HD / 8; ++ch) *chunk(ch) = make_uint4(0, 0, 0, 0);
              } else {
                __nv_bfloat162 acc = __float2bfloat162_rn(0.f);
#pragma unroll
                for (int ch = 0; ch < HD / 8; ++ch) gather_bad(acc, *chunk(ch));
                mine = __hisnan(acc.x) || __hisnan(acc.y);
                if (mine) {
#pragma unroll 1
                  for (int ch = 0; ch < HD / 8; ++ch) {
                    uint4 w = *chunk(ch);
                    w.x = zero_not_finite(w.x);
                    w.y = zero_not_finite(w.y);
                    w.z = zero_not_finite(w.z);
                    w.w = zero_not_finite(w.w);
                    *chunk(ch) = w;
                  }
                }
              }
            }
            const uint32_t keys = __ballot_sync(0xffffffffu, mine);
            if (lane == 0) noted[k0 / 32 + wg] = keys;
            odd |= mine;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          odd = ptx::named_bar_or(1 + x, GT, odd);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) {
          if (!early) ptx::mbar_arrive(&p_ready[2 * x]);
          ptx::mbar_arrive(&p_ready[2 * x + 1]);
        }
        // (group 0 noted them for both)
        late = odd || (nt == 2 && x == 1 && key0 + kStepT > plain_t) ? key0 : -1;
        if (late >= 0) {
          late_note = noted;
#pragma unroll
          for (int b = 0; b < 4; ++b) late_seen[b] = seen[b];
        }
      }
      if (ok && jobs > 0) {
        ok = __all_sync(0xffffffffu, wait(&pv_done[x], (nj - 1) & 1u));
        if (ok) ptx::tc_fence_after();
        if (ok) repair();
      }
      if (ptx::named_bar_or(5, GT * NG, !ok)) {
        ok = false;
        break;
      }
      // ---- the tile's rows ----
      float M = m_ref, L = l, fa = 1.f, fb = 0.f;            // weights of the two halves
      float* sB = reinterpret_cast<float*>(sQ);              // [128][HD], chunks of 4 swizzled
      if (NG == 2 && nt == 1) {
        if (x == 1) {
          sMl[row] = make_float2(m_ref, l);
          if (jobs > 0) {
#pragma unroll
            for (int b = 0; b < HD / 32; ++b) {
              uint32_t o[32];
              ptx::tmem_ld_32x32(aO + 32 * b, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(sB + row * HD + 4 * ((8 * b + j) ^ (row & 7))) =
                    make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
          }
        }
        ptx::named_bar_sync(5, GT * NG);
        if (x == 0) {
          const float2 ml = sMl[row];
          if (ml.y != 0.f) {
            M = fmaxf(m_ref, ml.x);
            fa = l != 0.f ? ex2(m_ref - M) : 0.f;
            fb = ex2(ml.x - M);
            L = fa * l + fb * ml.y;
          }
        }
      }
      const bool mine = nt == 2 || x == 0;                   // this group writes its rows
      const bool whole = n == pc.all;
      int c0 = 0, c1 = 0;
      if (!whole) paged_owners<Geo>(c, total, end - c.left - c.at, pc.all, &c0, &c1);
      // partials: [slot][NG][HD / 4][GT rows] of four columns, so that a warp's lanes
      // are neighbours in memory
      auto part_of = [&](int cc) { return ((size_t)cc * 2 + (cc == c0)) * NG + x; };
      const size_t slot = part_of(blockIdx.x);
      // The warp's 32 bf16 rows go out through shared memory, so that HD / 8
      // lanes write a row together: in the group's part of Q, or, a lane each, in
      // its row of the joined half, over columns that it has read.
      const int stage_ld = NG == 2 && nt == 1 ? HD * 4 : HD * 2;
      uint8_t* stage = sQ + warp * 32 * stage_ld;
      auto put = [&](int b, const float (&o)[32], float inv) {    // 32 columns of the row
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t w4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w4[e] = L == 0.f ? 0u : mmas::pack_bf16(o[8 * j + 2 * e] * inv, o[8 * j + 2 * e + 1] * inv);
          *reinterpret_cast<uint4*>(stage + lane * stage_ld + (((4 * b + j) ^ (lane & 7)) << 4)) =
              make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
      };
      auto send = [&]() {
        __syncwarp();
        const unsigned long long mine_to = reinterpret_cast<unsigned long long>(
            p.out + (long long)(rq.row0 + tok) * p.out_ld + (long long)head * HD);
        const unsigned on = __ballot_sync(0xffffffffu, live);
        constexpr int kLines = 256 / HD;
#pragma unroll 8
        for (int r0 = 0; r0 < 32; r0 += kLines) {
          const int rr = r0 + lane / (HD / 8), ch = lane % (HD / 8);
          uint4* to = reinterpret_cast<uint4*>(__shfl_sync(0xffffffffu, mine_to, rr)) + ch;
          const uint4 w = *reinterpret_cast<const uint4*>(stage + rr * stage_ld + ((ch ^ (rr & 7)) << 4));
          if ((on >> rr) & 1u) *to = w;
        }
      };
      if (mine && !dead) {
        const float inv = 1.f / L;
#pragma unroll 2
        for (int b = 0; b < HD / 32; ++b) {
          uint32_t u[32];
          ptx::tmem_ld_32x32(aO + 32 * b, u);
          ptx::tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = fa == 0.f ? 0.f : __uint_as_float(u[j]) * fa;
          if (fb != 0.f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 v = *reinterpret_cast<const float4*>(sB + row * HD + 4 * ((8 * b + j) ^ (row & 7)));
              o[4 * j] += fb * v.x;
              o[4 * j + 1] += fb * v.y;
              o[4 * j + 2] += fb * v.z;
              o[4 * j + 3] += fb * v.w;
            }
          }
          if (whole) {
            put(b, o, inv);
          } else if (live) {
            float4* po = reinterpret_cast<float4*>(p.part_o) + (slot * (HD / 4) + 8 * b) * GT + row;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              __stcg(po + j * GT, make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
          }
        }
        if (whole) send();
      }
      ptx::tc_fence_before();
      if (!whole && mine) {
        if (live) __stcg(p.part_ml + slot * GT + row, make_float2(M, L));
        if (p.cut) {
          if (tid == 0 && c0 == static_cast<int>(blockIdx.x))   // its first piece
            p.cut[c0] = {c1, rq.row0, tile0, nG, c.g * p.heads.G};
        } else {
          __threadfence();
          ptx::named_bar_sync(1 + x, GT);
          if (row == 0) s_last[x] = atomicAdd(p.arrive + NG * c0 + x, 1) == c1 - c0;
          ptx::named_bar_sync(1 + x, GT);
          if (s_last[x]) {
            __threadfence();
            if (row == 0) p.arrive[NG * c0 + x] = 0;            // for the next call
            if (!dead) {
              M = -CUDART_INF_F;
#pragma unroll 4
              for (int cc = c0; cc <= c1; ++cc) M = fmaxf(M, __ldcg(p.part_ml + part_of(cc) * GT + row).x);
              float o[HD] = {};
              L = 0.f;
              float2 ml = __ldcg(p.part_ml + part_of(c0) * GT + row);
              for (int cc = c0; cc <= c1; ++cc) {
                const float2 now = ml;
                if (cc < c1) ml = __ldcg(p.part_ml + part_of(cc + 1) * GT + row);
                const float f = now.y != 0.f ? ex2(now.x - M) : 0.f;
                L += f * now.y;
                const float4* src = reinterpret_cast<const float4*>(p.part_o) + part_of(cc) * (HD / 4) * GT + row;
#pragma unroll
                for (int j = 0; j < HD / 4; ++j) {
                  const float4 v = __ldcg(src + j * GT);
                  if (now.y != 0.f) {
                    o[4 * j] += f * v.x;
                    o[4 * j + 1] += f * v.y;
                    o[4 * j + 2] += f * v.z;
                    o[4 * j + 3] += f * v.w;
                  }
                }
              }
#pragma unroll
              for (int b = 0; b < HD / 32; ++b) put(b, reinterpret_cast<float(&)[32]>(o[32 * b]), 1.f / L);
              send();
            }
          }
        }
      }
      it += 2 * kPer * n;
      // the rows on their way out lie where the next tile's queries go
      ptx::named_bar_sync(5, GT * NG);
    }
    if (!ok) fail();
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kIssue) {
    __syncwarp();
    ptx::tmem_dealloc(tbase, S::kTmem);
  }
}

// Joins the tiles that shares' borders cut, each 32 rows (a lane to a row) to a block of
// eight warps, which share out the parts for the weights and the columns for the sums.
// Blocks x: the CTA that holds a tile's first piece.  (32 warps to a block, a warp for
// four columns, took longer: 128 rows over 4096 slots 32 us against 27.)
template <int HD, int NG>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedAttnParams p) {
  constexpr int GT = Tc<HD, NG>::kGroup, kRound = 64, kFours = HD / 4, kCols = kFours / 8;
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

template <int HD, int NG>
dflash_status launch_tc(PagedAttnParams p, const dflash_pages& pages, cudaStream_t st) {
  using S = Tc<HD, NG>;
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(paged_attn_tc_kernel<HD, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  PagedTcMaps maps;
  const int rows = pages.n_pages * pages.n_kv * pages.page_size;
  const int box = pages.page_size < S::kKeys ? pages.page_size : S::kKeys;
  if (!encode_kmajor_map(&maps.k, pages.k, rows, HD, HD, box) ||
      !encode_kmajor_map(&maps.v, pages.v, rows, HD, HD, box))
    return set_error(DFLASH_ERR_CUDA, "paged attention: cannot encode the TMA descriptors");
  const int grid = num_sms() * S::kPerSm;
  // A few parts to a tile are joined by the last CTA to arrive, which costs no launch
  // and hides behind the others' work; many by a kernel of their own, since one CTA
  // reads a part in about 2 us.  Measured, by a kernel / by the last CTA, us: 16 rows over
  // 8192 slots (38 parts) 27 / 45, 128 over 4096 (19) 30 / 37; trees of 129, 257, 385 and
  // 513 rows over 8192 (6.3, 3.8, 2.7, 2.1) 40 / 45, 55.5 / 56.1, 70 / 69, 84 / 82; 6, 9,
  // 10, 12 and 16 chains of 16 over 4096 (6.3, 4.2, 3.8, 3.2, 2.4) 34 / 37, 42.1 / 42.4,
  // 44.4 / 46.4, 49 / 51, 59.5 / 59.9; a prompt chunk (1.6) 243 / 235.  (They meet
  // between two and three parts in 64-row tiles, at three in 256-row ones; the rule's
  // four costs 2 us at most.)
  const long long tiles = (p.n_rows * (long long)p.heads.G + S::kRows - 1) / S::kRows * p.pv.n_kv;
  if (tiles * 4 >= grid) p.cut = nullptr;
  {
    TraceScope ts("paged_attn_tc", st);
    launch_k(paged_attn_tc_kernel<HD, NG>, dim3(grid), dim3(S::kThreads), S::kBytes, st, maps, p);
  }
  if (p.cut) {
    TraceScope ts("paged_join", st);
    launch_k(paged_join_kernel<HD, NG>, dim3(grid, S::kRows / 32), dim3(256), 0, st, p);
  }
  return DFLASH_OK;
}

// Header, arrival counters, (max, sum) pairs, partial rows.
struct PagedWs {
  size_t arrive, cut, ml, o, bytes;
};
// Every kernel: two CTAs an SM at most, two counters an SM, and for each SM two
// slots of 256 rows (or 2 x 2 of 128, or of 16).
PagedWs paged_ws(int sms, int head_dim) {
  PagedWs w;
  const size_t rows = (size_t)sms * 2 * 256;
  w.arrive = 256;
  w.cut = w.arrive + align_up((size_t)sms * 2 * sizeof(int), 256);
  w.ml = w.cut + align_up((size_t)sms * 2 * sizeof(PagedCut), 256);
  w.o = w.ml + align_up(rows * sizeof(float2), 256);
  w.bytes = w.o + rows * head_dim * sizeof(float);
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
  const dflash_status s = check_pages(pages, n_req, "paged attention", &p.pv);
  if (s) return s;
  const int hd = pages->head_dim;
  if (pages->dtype != DFLASH_BF16)
    return set_error(DFLASH_ERR_UNSUPPORTED, "paged attention: the cache must be bf16");
  DFL_REQUIRE(n_req >= 0 && n_rows >= 0 && max_rows >= 0, "paged attention: sizes must be >= 0");
  DFL_REQUIRE(n_q >= pages->n_kv && n_q % pages->n_kv == 0,
              "paged attention: n_q must be a multiple of n_kv");
  DFL_REQUIRE((long long)n_rows * n_q < (1ll << 30), "paged attention: rows x heads exceed 2^30");
  DFL_REQUIRE(q_ld >= (long long)n_q * hd && out_ld >= (long long)n_q * hd && q_ld % 8 == 0 &&
                  out_ld % 8 == 0,
              "paged attention: row strides too small or not multiples of 8");
  DFL_REQUIRE(mask == nullptr || (mask_ld >= 1 && (long long)mask_ld * 32 >= max_rows),
              "paged attention: mask rows shorter than max_rows");
  if (n_req == 0 || n_rows == 0) return DFLASH_OK;
  DFL_REQUIRE(row_off && pos0 && q && out, "paged attention: null pointer argument");
  DFL_REQUIRE(((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) == 0,
              "paged attention: q and out must be 16-byte aligned");
  const PagedWs w = paged_ws(num_sms(), hd);
  if (!ws || ws_bytes < w.bytes)
    return set_error(DFLASH_ERR_WORKSPACE, "paged attention workspace needs %zu bytes, got %zu",
                     w.bytes, ws_bytes);
  DFL_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 15) == 0,
              "paged attention: the workspace must be 16-byte aligned");
  p.n_req = n_req;
  p.n_rows = n_rows;
  p.heads.G = n_q / pages->n_kv;
  p.heads.m = static_cast<uint32_t>((1ull << 32) / p.heads.G);
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
  p.cut = reinterpret_cast<PagedCut*>(b + w.cut);
  p.status = reinterpret_cast<int*>(b);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // The smallest tile that takes all rows of a (request, KV head): keys and values
  // are then read once.  Measured, us: one token of 32 requests in 16-row tiles 99, in
  // 64-row tiles 108; of one request over 2048 slots 10 and 36.  64 rows of 32 requests in
  // 64-row tiles 110, in 256-row tiles 138; 128 rows of 19 requests over 4064 slots 65 in
  // 256-row tiles, 91 in 128-row tiles of which two share an SM.
  const long long rows = (long long)max_rows * p.heads.G;
  dflash_status e = DFLASH_OK;
  if (rows <= kRowsS)
    hd == 128 ? launch_small<128>(p, st) : launch_small<64>(p, st);
  else if (rows <= Tc<128, 1>::kRows)
    e = hd == 128 ? launch_tc<128, 1>(p, *pages, st) : launch_tc<64, 1>(p, *pages, st);
  else
    e = hd == 128 ? launch_tc<128, 2>(p, *pages, st) : launch_tc<64, 2>(p, *pages, st);
  if (e) return e;
  return check_launch("paged attention");
}

}  // extern "C"
