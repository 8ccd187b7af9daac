// Attention of new tokens over a paged KV cache held in 8 bits.
//
// "Accelerating Speculative Decoding with Block Diffusion Draft Trees", section
// 3.4.5, over a cache of e4m3 codes with a power-of-two scale for each block of 16
// slots of a KV head: with key codes c_t, value codes d_t and their blocks' exponents
// a, b, per (row, head)
//
//   s_t = q . c_t 2^a / sqrt(hd),   out = sum_t 2^(s_t - m) 2^b d_t / sum_t 2^(s_t - m)
//
// (s in base-2 units).  Codes are exact in fp16, so both products run on fp16 tensor
// cores with the codes as they are: the key's scale multiplies the fp32 score, the
// value's goes into the exponent of the weight, 2^((s_t - m) + b - r).  m is the running
// maximum of s_t and r that of (s_t - m) + b: the largest term of either sum is near 1
// whatever the blocks' scales are, so weights keep fp16's 11 bits (and lose only what
// is below 2^-24 of the largest).  A row of q is taken to fp16 at a power of two at which
// its largest element is near 2^15: bf16's 8 bits are kept exactly down to 2^-32 of it.
//
// The work is shared out as in paged_attention.h.
#include <cmath>

#include <math_constants.h>

#include "gemm.h"
#include "kernels.h"
#include "paged_attention.h"
#include "ptx.cuh"

namespace dfl {

namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull, kMaxLimitNs = 60000000000ull;

struct PagedE4M3Params : PagedAttnParams {
  const uint8_t *k_scale, *v_scale;
};

// Pools as lines of 128 bytes, box: 16 slots, 128-byte swizzle.
struct PagedE4M3Maps {
  CUtensorMap k, v;
};

// Two codes (the low or the high half of a word) as two fp16.
__device__ __forceinline__ uint32_t half2_lo(uint32_t codes) {
  uint32_t h;
  asm("{.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(h) : "r"(codes));
  return h;
}
__device__ __forceinline__ uint32_t half2_hi(uint32_t codes) {
  uint32_t h;
  asm("{.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;}" : "=r"(h) : "r"(codes));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of fp16, rows on groups of four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t h) {
  uint32_t t;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(h));
  return t;
}

// 2^(b - 127) of a scale's byte (255, which no append writes, as 254).
__device__ __forceinline__ float scale_of(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(min(b, 254u) << 23);
}

// A word's codes that are NaN, as 0xFF bytes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t top = (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
  return top * 0xFFu;
}

// ---------------------------------------------------------------------------
// Few query rows (decoding): tiles of 8 NT rows on warp-level MMAs.
// ---------------------------------------------------------------------------
// Four warps; a step is 64 keys, a block of 16 to each warp, which keeps its own ring of
// blocks (TMA, kStagesS deep) and its own running softmax, so the main loop has no block
// barrier.  The products are transposed, S^T = K Q^T and O^T = V^T P^T: the codes are the
// A operand, 16 keys or 16 columns at a time, and 8 query rows fill an MMA, where rows on
// the other side would leave half of 16 idle for the usual four or eight heads to a
// KV head.  Which key, column or element a lane holds is free as long as both operands
// agree: a lane reads its codes as 16-byte pieces of a slot, and turns them into fragments
// by conversion alone (and, for V, a byte permutation that pairs two slots).
constexpr int kStepS = 64, kStagesS = 6, kThreadsS = 128, kPerSmS = 2;

template <int NT>
using GeoS = PagedGeo<8 * NT, kStepS, 4, 8 * NT, 2>;

template <int HD, int NT>
struct Small {
  static constexpr int kTile = 16 * HD;                           // a block of K or V
  static constexpr int kRing = 4 * kStagesS * 2 * kTile;
  static constexpr int kRows = 8 * NT, kLd = HD + 8;
  static constexpr int kMl = kRing, kBar = kMl + 4 * kRows * 8, kBytes = kBar + 4 * kStagesS * 8 + 16;
  static_assert(4 * kRows * kLd * 4 <= kRing, "the warps' states meet in the idle ring");
};

template <int HD, int NT>
__global__ void __launch_bounds__(kThreadsS, kPerSmS)
paged_attn_small_e4m3_kernel(const __grid_constant__ PagedE4M3Maps maps, const PagedE4M3Params p) {
  using S = Small<HD, NT>;
  using Geo = GeoS<NT>;
  constexpr int kLines = HD / 8;               // 128-byte lines of a block
  constexpr int kW = HD / 16;                  // MMA steps of q . k
  constexpr int kT = HD / 16;                  // column tiles of O^T
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ra = lane >> 2, cq = lane & 3;     // fragment row (and + 8), and column pair
  uint8_t* ring = smem + warp * (kStagesS * 2 * S::kTile);
  float* sO = reinterpret_cast<float*>(smem);                          // [4][kRows][kLd], in the ring
  float2* sMl = reinterpret_cast<float2*>(smem + S::kMl);              // [4][kRows]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBar) + warp * kStagesS;
  int* sLast = reinterpret_cast<int*>(smem + S::kBar + 4 * kStagesS * 8);
  if (ptx::smem_addr(smem) & 1023) {                                   // (the swizzle counts on it)
    record_status(p.status, DFLASH_ERR_UNSUPPORTED);
    return;
  }
  if (lane == 0) {
    for (int s = 0; s < kStagesS; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&maps.k);
    ptx::prefetch_tmap(&maps.v);
  }
  __syncwarp();

  pdl_wait();
  pdl_trigger();
  long long total, end;                                  // the line, and the end of this CTA's share
  PagedCursor c;
  const uint64_t header = *reinterpret_cast<const volatile uint64_t*>(p.status + 2);
  paged_plan<Geo>(p, lane, &total, &end, &c);
  const uint64_t limit = header == 0 || header > kMaxLimitNs ? kTimeoutNs : header;
  const uint64_t pol = ptx::policy_evict_first();
  const int nowhere = ((p.pv.n_pages * p.pv.n_kv) << p.pv.page_shift) / kScaleBlock * kLines;   // past the pool: zeros
  uint32_t asked = 0, had = 0;                           // blocks of this warp's ring
  bool ok = true;

  for (PagedPiece pc; c.left > 0; paged_next<Geo>(p, pc, &c)) {
    pc = PagedPiece::of<Geo>(c);
    if (pc.n <= 0) continue;
    const PagedReq rq = c.rq;
    const int nG = rq.n * p.heads.G, rho0 = c.j * S::kRows;
    const int kend = rq.key_end<Geo>(c.j, p.heads);
    const int n = pc.n;
    const int k0 = pc.first * kStepS + warp * 16;   // this warp's first key of the piece
    const int head0 = c.g * p.heads.G;

    // Lane i looks up the blocks of steps i, i + 32, ...: the line in the pool and the two
    // scales, a round of 32 steps ahead.
    bool missing = false;
    struct Round {
      int line;
      uint32_t scales;
    };
    auto look = [&](int i0) {
      const int t = k0 + (i0 + lane) * kStepS;
      Round x = {nowhere, 127u | 127u << 8};
      if (i0 + lane < n && t < kend) {
        const int page = page_of(p.pv, c.r, t);
        missing |= page < 0;
        if (page >= 0) {
          const int b = static_cast<int>(pool_row(p.pv, page, c.g, t) / kScaleBlock);
          x.line = b * kLines;
          x.scales = __ldg(p.k_scale + b) | static_cast<uint32_t>(__ldg(p.v_scale + b)) << 8;
        }
      }
      return x;
    };
    Round now = look(0), next = look(32);
    // steps whose keys lie before the tile's end
    const int steps = kend > k0 ? min(n, (kend - k0 + kStepS - 1) / kStepS) : 0;
    auto load = [&](int i, int round0) {                 // the block of step i, round0 <= i < round0 + 64
      if (i >= steps || !ok) return;
      const int a = __shfl_sync(0xffffffffu, now.line, i & 31), b = __shfl_sync(0xffffffffu, next.line, i & 31);
      const int line = i < round0 + 32 ? a : b, s = asked % kStagesS;
      if (lane == 0) {
        uint8_t* dst = ring + s * 2 * S::kTile;
        ptx::mbar_arrive_expect_tx(&full[s], 2 * S::kTile);
        ptx::tma_load_2d(dst, &maps.k, &full[s], 0, line, pol);
        ptx::tma_load_2d(dst + S::kTile, &maps.v, &full[s], 0, line, pol);
      }
      ++asked;
    };
#pragma unroll
    for (int i = 0; i < kStagesS - 1; ++i) load(i, 0);

    // q: row 8 nt + ra, of which the lane holds HD / 4 neighbours; its power of two, and the
    // score's factor of rows 2 cq, 2 cq + 1
    uint32_t qf[NT][kW][2];
    float f[NT][2];
    int tok[NT][2], lim[NT][2];                          // their token, and the first slot past what they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rho = rho0 + 8 * nt + ra;
      const bool live = rho < nG;
      const int to = live ? p.heads.quot(rho) : 0;
      const __nv_bfloat16* row = p.q + (long long)(rq.row0 + to) * p.q_ld +
                                 (long long)(head0 + (live ? rho - to * p.heads.G : 0)) * HD + cq * (HD / 4);
      uint32_t w[HD / 8];
#pragma unroll
      for (int i = 0; i < HD / 32; ++i) {
        const uint4 u = live ? __ldg(reinterpret_cast<const uint4*>(row) + i) : make_uint4(0, 0, 0, 0);
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max(static_cast<int>(top >> 7), 16);          // its biased exponent
      const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);        // 2^(141 - e)
      const float down = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        const float lo = __uint_as_float(w[i] << 16) * up, hi = __uint_as_float(w[i] & 0xFFFF0000u) * up;
        qf[nt][i >> 1][i & 1] = pack_f16(lo, hi);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f[nt][h] = __shfl_sync(0xffffffffu, down, (2 * cq + h) * 4);
        const int rho_h = rho0 + 8 * nt + 2 * cq + h;
        tok[nt][h] = rho_h < nG ? p.heads.quot(rho_h) : 0;
        lim[nt][h] = rho_h < nG ? min(rq.p0 + (rq.masked ? 0 : tok[nt][h] + 1), kend) : 0;
      }
    }
    // keys below `plain` are seen by every row of the tile
    const int plain = min(rq.masked ? rq.p0 : rq.p0 + p.heads.quot(rho0) + 1, kend);

    float o[NT][kT][4] = {};
    float m[NT][2], r[NT][2], l[NT][2];                  // running maxima (of s, of s - m + b), sum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[nt][h] = r[nt][h] = -CUDART_INF_F;
        l[nt][h] = 0.f;
      }
    for (int i = 0, round0 = 0; i < steps; ++i) {
      if (i == round0 + 32) {
        round0 = i;
        now = next;
        next = look(i + 32);
      }
      load(i + kStagesS - 1, round0);
      const uint32_t s = had % kStagesS;
      if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(&full[s], had / kStagesS & 1u, limit, nullptr));
      if (!ok) break;
      ++had;
      const int t0 = k0 + i * kStepS;
      const uint8_t* sK = ring + s * 2 * S::kTile;
      const uint8_t* sV = sK + S::kTile;
      const uint32_t scales = __shfl_sync(0xffffffffu, now.scales, i & 31);
      // piece ch (16 bytes) of a slot
      auto piece = [&](const uint8_t* tile, int slot, int ch) {
        if constexpr (HD == 128) return tile + slot * 128 + ((ch ^ (slot & 7)) << 4);
        return tile + (slot >> 1) * 128 + (((((slot & 1) << 2) + ch) ^ ((slot >> 1) & 7)) << 4);
      };
      // S^T
      float st[NT][4] = {};
#pragma unroll
      for (int u = 0; u < HD / 64; ++u) {
        const uint4 ka = *reinterpret_cast<const uint4*>(piece(sK, ra, HD / 64 * cq + u));
        const uint4 kb = *reinterpret_cast<const uint4*>(piece(sK, ra + 8, HD / 64 * cq + u));
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a[4] = {half2_lo(wa[j]), half2_lo(wb[j]), half2_hi(wa[j]), half2_hi(wb[j])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(st[nt], a, qf[nt][4 * u + j][0], qf[nt][4 * u + j][1]);
        }
      }
      const bool all = t0 + 16 <= plain;                 // warp-uniform
      const float ks = scale_of(scales & 0xFFu);
      const float b = static_cast<float>(static_cast<int>(scales >> 8)) - 127.f;
      uint32_t seen = 0;                                 // bit 4 nt + e of st[nt][e] (where not all are)
      float mx[NT][2];
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e & 1;
          st[nt][e] *= fminf(f[nt][h] * ks, 0x1p90f);    // (no infinity times zero)
          if (!all) {
            const int t = t0 + ra + 8 * (e >> 1);
            bool see = t < lim[nt][h];
            if (rq.masked && !see && t >= rq.p0 && t < kend && rho0 + 8 * nt + 2 * cq + h < nG) {
              const int at = t - rq.p0;
              see = (at >> 5) < p.mask_ld &&
                    ((__ldg(p.mask + (size_t)(rq.row0 + tok[nt][h]) * p.mask_ld + (at >> 5)) >> (at & 31)) & 1u);
            }
            if (see) seen |= 1u << (4 * nt + e);
            else st[nt][e] = -CUDART_INF_F;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x = fmaxf(st[nt][h], st[nt][h + 2]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          mx[nt][h] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          raise |= mx[nt][h] > m[nt][h] + kLazy || mx[nt][h] - m[nt][h] + b > r[nt][h] + kLazy;
        }
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (mx[nt][h] == -CUDART_INF_F) continue;
            const float m2 = fmaxf(m[nt][h], mx[nt][h]), was = m[nt][h] - m2 + r[nt][h];
            const float r2 = fmaxf(was, mx[nt][h] - m2 + b), g = ex2(was - r2);
            l[nt][h] *= ex2(m[nt][h] - m2);
            m[nt][h] = m2;
            r[nt][h] = r2;
#pragma unroll
            for (int j = 0; j < kT; ++j) {
              o[nt][j][h] *= g;
              o[nt][j][h + 2] *= g;
            }
          }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e & 1;
          const bool none = m[nt][h] == -CUDART_INF_F;
          const float x = st[nt][e] - (none ? 0.f : m[nt][h]);
          l[nt][h] += ex2(x);
          w[e] = ex2(x + (none ? 0.f : b - r[nt][h]));
        }
        pf[nt][0] = transpose8(pack_f16(w[0], w[1]));
        pf[nt][1] = transpose8(pack_f16(w[2], w[3]));
      }
      // V: slots 2 cq, + 1, + 8, + 9, columns HD / 8 * ra ..
      uint32_t v[4][HD / 32];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int slot = 2 * cq + (k & 1) + 8 * (k >> 1);
        if constexpr (HD == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(piece(sV, slot, ra));
          v[k][0] = u.x;
          v[k][1] = u.y;
          v[k][2] = u.z;
          v[k][3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(piece(sV, slot, ra >> 1) + (ra & 1) * 8);
          v[k][0] = u.x;
          v[k][1] = u.y;
        }
      }
      if (!all) {
        // A NaN that some row may not see (0 * NaN is not 0): it counts as zero in the
        // product, and the rows that see it become NaN in its column.
        uint32_t any = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < HD / 32; ++j) any |= nan_bytes(v[k][j]);
        if (__any_sync(0xffffffffu, any != 0)) {
#pragma unroll 1
          for (int key = 0; key < 16; ++key) {
            const int from = (lane & ~3) | ((key & 7) >> 1), k = (key & 1) + 2 * (key >> 3);
            const uint32_t sb = __shfl_sync(0xffffffffu, seen, ((key & 7) << 2) | cq) >> (2 * (key >> 3));
#pragma unroll
            for (int j = 0; j < HD / 32; ++j) {
              const uint32_t mine = k == 0 ? v[0][j] : k == 1 ? v[1][j] : k == 2 ? v[2][j] : v[3][j];
              // (which lane's word it is goes by the key: the same k in all lanes)
              const uint32_t bad = nan_bytes(__shfl_sync(0xffffffffu, mine, from));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 8; ++e)                // column 4 j + e / 2 of the lane's, row 2 cq + e % 2
                  if (((sb >> (4 * nt + (e & 1))) & 1u) && ((bad >> (8 * (e >> 1))) & 1u))
                    o[nt][2 * j + (e >> 2)][((e >> 1) & 1) * 2 + (e & 1)] = CUDART_NAN_F;
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < HD / 32; ++j) v[k][j] &= ~nan_bytes(v[k][j]);
        }
      }
      // O^T
#pragma unroll
      for (int j = 0; j < HD / 32; ++j) {
        const uint32_t x0 = __byte_perm(v[0][j], v[1][j], 0x5140), x1 = __byte_perm(v[0][j], v[1][j], 0x7362);
        const uint32_t y0 = __byte_perm(v[2][j], v[3][j], 0x5140), y1 = __byte_perm(v[2][j], v[3][j], 0x7362);
        const uint32_t a0[4] = {half2_lo(x0), half2_hi(x0), half2_lo(y0), half2_hi(y0)};
        const uint32_t a1[4] = {half2_lo(x1), half2_hi(x1), half2_lo(y1), half2_hi(y1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(o[nt][2 * j], a0, pf[nt][0], pf[nt][1]);
          mma_f16(o[nt][2 * j + 1], a1, pf[nt][0], pf[nt][1]);
        }
      }
      __syncwarp();   // the slot may be loaded again
    }

    if (__any_sync(0xffffffffu, missing))
      for (int t0 = k0; t0 < min(k0 + n * kStepS, kend); t0 += kStepS)
        if (page_of(p.pv, c.r, t0) < 0 && paged_seen<Geo>(p, c, t0, min(t0 + 16, kend), lane) && lane == 0)
          record_status(p.status, DFLASH_ERR_INVALID_ARG);
    if (warp == 0) paged_past<Geo>(p, c, lane);

    // every copy lands before the ring is used for the states, or the CTA exits
    if (!ok && lane == 0) record_status(p.status, DFLASH_ERR_TIMEOUT);
    for (; had < asked; ++had)
      ptx::mbar_wait_bounded(&full[had % kStagesS], had / kStagesS & 1u, kTimeoutNs, nullptr);

    // the four warps' states, of the tile's live rows; O with m as its reference too
    const int live = min(S::kRows, nG - rho0);
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], x);
        const int row = 8 * nt + 2 * cq + h;
        if (row >= live) continue;
        const float g = m[nt][h] == -CUDART_INF_F ? 1.f : ex2(r[nt][h]);
        float* dst = sO + (warp * S::kRows + row) * S::kLd + HD / 8 * ra;
#pragma unroll
        for (int j = 0; j < kT; j += 2)
          *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[nt][j][h] * g, o[nt][j][h + 2] * g,
                                                                o[nt][j + 1][h] * g, o[nt][j + 1][h + 2] * g);
        if (ra == 0) sMl[warp * S::kRows + row] = make_float2(m[nt][h], l[nt][h]);
      }
    __syncthreads();
    paged_finish_small<HD, S::kRows, S::kLd, kThreadsS, Geo>(p, c, pc, total, end, rho0, live, sO, sMl, smem, sLast);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();                                     // the ring is free again
  }
}

template <int HD, int NT>
dflash_status launch_small(const PagedE4M3Params& p, const dflash_pages_e4m3& pages, cudaStream_t st) {
  using S = Small<HD, NT>;
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(paged_attn_small_e4m3_kernel<HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  PagedE4M3Maps maps;
  const int lines = pages.n_pages * pages.n_kv * (pages.page_size / kScaleBlock) * (HD / 8);
  if (!encode_kmajor_map(&maps.k, pages.k, lines, 64, 64, HD / 8) ||       // (lines as 64 elements of 16 bits)
      !encode_kmajor_map(&maps.v, pages.v, lines, 64, 64, HD / 8))
    return set_error(DFLASH_ERR_CUDA, "paged attention e4m3: cannot encode the TMA descriptors");
  TraceScope ts("paged_attn_small_e4m3", st);
  launch_k(paged_attn_small_e4m3_kernel<HD, NT>, dim3(num_sms() * kPerSmS), dim3(kThreadsS), S::kBytes, st, maps, p);
  return DFLASH_OK;
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" {

size_t dflash_paged_attention_e4m3_workspace_bytes(int n_q, int n_kv, int head_dim) {
  if (n_kv < 1 || n_q < n_kv || n_q % n_kv || (head_dim != 64 && head_dim != 128)) return 0;
  return paged_ws(num_sms(), head_dim).bytes;
}

dflash_status dflash_paged_attention_e4m3(const dflash_pages_e4m3* pages, int n_req, int n_rows,
                                          int n_q, const int32_t* row_off, const int32_t* pos0,
                                          int max_rows, const void* q, long long q_ld,
                                          const uint32_t* mask, int mask_ld, void* out,
                                          long long out_ld, void* ws, size_t ws_bytes,
                                          void* stream) {
  PagedE4M3Params p{};
  const dflash_status s = check_pages(pages, n_req, "paged attention e4m3", &p.pv);
  if (s) return s;
  const int hd = pages->head_dim;
  DFL_REQUIRE(n_req >= 0 && n_rows >= 0 && max_rows >= 0, "paged attention e4m3: sizes must be >= 0");
  DFL_REQUIRE(n_q >= pages->n_kv && n_q % pages->n_kv == 0,
              "paged attention e4m3: n_q must be a multiple of n_kv");
  DFL_REQUIRE((long long)n_rows * n_q < (1ll << 30), "paged attention e4m3: rows x heads exceed 2^30");
  DFL_REQUIRE(q_ld >= (long long)n_q * hd && out_ld >= (long long)n_q * hd && q_ld % 8 == 0 &&
                  out_ld % 8 == 0,
              "paged attention e4m3: row strides too small or not multiples of 8");
  DFL_REQUIRE(mask == nullptr || (mask_ld >= 1 && (long long)mask_ld * 32 >= max_rows),
              "paged attention e4m3: mask rows shorter than max_rows");
  if (n_req == 0 || n_rows == 0) return DFLASH_OK;
  DFL_REQUIRE(row_off && pos0 && q && out, "paged attention e4m3: null pointer argument");
  DFL_REQUIRE(((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) == 0,
              "paged attention e4m3: q and out must be 16-byte aligned");
  const PagedWs w = paged_ws(num_sms(), hd);
  if (!ws || ws_bytes < w.bytes)
    return set_error(DFLASH_ERR_WORKSPACE, "paged attention e4m3 workspace needs %zu bytes, got %zu",
                     w.bytes, ws_bytes);
  DFL_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 15) == 0,
              "paged attention e4m3: the workspace must be 16-byte aligned");
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
  p.k_scale = pages->k_scale;
  p.v_scale = pages->v_scale;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long rows = (long long)max_rows * p.heads.G;
  dflash_status e;
  if (rows <= 8)
    e = hd == 128 ? launch_small<128, 1>(p, *pages, st) : launch_small<64, 1>(p, *pages, st);
  else
    e = hd == 128 ? launch_small<128, 2>(p, *pages, st) : launch_small<64, 2>(p, *pages, st);
  if (e) return e;
  return check_launch("paged attention e4m3");
}

}  // extern "C"
