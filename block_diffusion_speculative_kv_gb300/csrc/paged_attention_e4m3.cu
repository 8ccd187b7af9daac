// Attention of new tokens over a paged KV cache held in 8 bits.
//
// "Accelerating Speculative Decoding with Block Diffusion Draft Trees", section
// 3.4.5, over a cache of e4m3 codes with a power-of-two scale for each block of 16
// slots of a KV head: with key codes c_t, value codes d_t and their blocks' exponents
// a, b, per (row, head)
//
//   s_t = q . c_t 2^a / sqrt(hd),   out = sum_t 2^(s_t - m) 2^b d_t / sum_t 2^(s_t - m)
//
// (s in base-2 units).  Codes enter both products as they are, as fp16 (exact) or as e4m3:
// the key's scale multiplies the fp32 score, the value's goes into the exponent of the
// weight, 2^((s_t - m) + b - r).  m is the running maximum of s_t and r that of
// (s_t - m) + b: the largest term of either sum is near 1 whatever the blocks' scales are,
// so fp16 weights keep their 11 bits (and lose only what is below 2^-24 of the largest).
// A row of q is scaled by a power of two of its own: to fp16, its largest element near
// 2^15, which keeps bf16's 8 bits exactly down to 2^-32 of it; or to two e4m3 codes.
//
// The work is shared out as in paged_attention.h.
#include <cmath>

#include <cuda_fp8.h>
#include <math_constants.h>

#include "gemm.h"
#include "kernels.h"
#include "paged_attention.h"
#include "ptx.cuh"

namespace dfl {

namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull, kMaxLimitNs = 60000000000ull;

// How far the references of a row's weights may lag behind their maxima (base-2 units):
// weights up to 2^14 fit fp16, and a reference that lags loses nothing below.
constexpr float kLag = 14.f;

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

// 2^(b - 127) of a scale's byte, and b - 127.
__device__ __forceinline__ float scale_of(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(min(b, static_cast<uint32_t>(kTopScale)) << 23);
}
__device__ __forceinline__ float exponent_of(uint32_t b) {
  return static_cast<float>(min(static_cast<int>(b), kTopScale) - 127);
}

// 2^x of a row's r, -127 at least: ex2 alone would make zero of what is below 2^-126.
__device__ __forceinline__ float ex2_low(float x) {
  const bool low = x < -64.f;
  return ex2(low ? x + 64.f : x) * (low ? 0x1p-64f : 1.f);
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
// HBM bounds it: 32 single tokens over 512 .. 8192 slots take 57 us, 5.5 TB/s of 6.8 (of the
// 16-bit cache 100), the tail of shares and the chain of conversions, MMAs and exponentials
// in each warp the rest.  CTAs an SM and stages, us: 2 and 6 64, 3 and 4 58, 4 and 3 60, 3 and
// 3 57.  One request over 2048 slots takes 11 (launch, plan, two steps, join; the 16-bit cache
// 10), over 8192 17 (15), over 65536 37 (52), over 131072 53 (90).
constexpr int kStepS = 64, kStagesS = 3, kThreadsS = 128, kPerSmS = 3;

template <int NT>
using GeoS = PagedGeo<8 * NT, kStepS, 4, 8 * NT, 2>;

template <int HD, int NT>
struct Small {
  static constexpr int kTile = 16 * HD;                           // a block of K or V
  static constexpr int kRing = 4 * kStagesS * 2 * kTile;
  static constexpr int kRows = 8 * NT, kLd = HD + 8, kPairs = paged_pairs(kRows, kPerSmS);
  static constexpr int kMl = kRing > kPairs ? kRing : kPairs;     // (the join's pairs lie over the ring)
  static constexpr int kBar = kMl + 4 * kRows * 8, kBytes = kBar + 4 * kStagesS * 8 + 16;
  static_assert(kPerSmS * (kBytes + 1024) <= 228 * 1024, "shared memory of an SM");
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
      const float b = exponent_of(scales >> 8);
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
          raise |= mx[nt][h] > m[nt][h] + kLag || mx[nt][h] - m[nt][h] + b > r[nt][h] + kLag;
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
        const float g = m[nt][h] == -CUDART_INF_F ? 1.f : ex2_low(r[nt][h]);
        float* dst = sO + (warp * S::kRows + row) * S::kLd + HD / 8 * ra;
#pragma unroll
        for (int j = 0; j < kT; j += 2)
          *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[nt][j][h] * g, o[nt][j][h + 2] * g,
                                                                o[nt][j + 1][h] * g, o[nt][j + 1][h + 2] * g);
        if (ra == 0) sMl[warp * S::kRows + row] = make_float2(m[nt][h], l[nt][h]);
      }
    __syncthreads();
    paged_finish_small<HD, S::kRows, S::kLd, kThreadsS, S::kMl, kPerSmS, Geo>(p, c, pc, total, end, rho0, live, sO, sMl,
                                                                              smem, sLast);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();                                     // the ring is free again
  }
}

template <int HD, int NT>
dflash_status launch_small(const PagedE4M3Params& p, const dflash_pages_e4m3& pages, cudaStream_t st) {
  using S = Small<HD, NT>;
  static_assert(kPerSmS <= kMostCtas && kPerSmS * S::kRows <= 256, "the workspace's counters and slots");
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

// ---------------------------------------------------------------------------
// Many query rows (chains, trees, prompt chunks): tensor-core tiles.
// ---------------------------------------------------------------------------
// The tiles, the turns of the softmax groups and the joins are those of the 16-bit
// cache's kernel (paged_attention.cu): NG MMA tiles of 128 query rows (NG = 1: 64 rows, two
// CTAs to an SM) against steps of 128 keys, S_x and O_x in TMEM, P_x over S_x as the A
// operand of P V.  What differs:
//   Q K^T  takes the key codes as TMA brings them, on the e4m3 cores: a row of q is the
//     sum of two codes, hi + lo, at a power of two at which its largest element lies in
//     [128, 256).  bf16's 8 bits are two codes' 4 + 4, so that is exact for elements down
//     to 2^-10 of the row's largest, and off by 2^-17 of the largest below.  Twice the
//     products at twice the rate: the time of the 16-bit form, and no conversion of K.
//   P V    runs in fp16, since e4m3's 4 bits of P would not do: warps of their own turn
//     the value codes into an fp16 tile in shared memory, laid out as TMA would, while
//     the softmax of the step runs.  The last steps of a tile, where some row may not see
//     some key, are also looked through for NaN: such a code counts as zero, its key is
//     noted, and rows that see it become NaN in its column.
//   scales come with the loads, 8 + 8 to a step, and are applied as in the small tiles:
//     a key block's to its 16 scores, a value block's in the exponent of its 16 weights,
//     2^((s - m) + b - r), and the sum l takes each 16's sum back at 2^(r - b).
// A row has two threads, each with half of a step's keys and of O's columns: their registers
// hold 64 scores where one thread's would hold 128 (a prompt chunk of 2048 rows over 8192 slots
// 289 against 386 us, and 314 with 216 registers to a thread), and the halves' P V start apart.
// References lag: m and r move only when a weight would pass 2^kLag.  What bounds it is
// the chain scores - softmax - P V of each group, as in the 16-bit cache's kernel, with
// conversion beside it: the chunk takes 289 us (1.07 PFLOP/s; tensor pipe 46% busy, issue slots
// 51%).  When it took 308, it took 288 without the conversion of V, 289 without exponentials,
// 297 with one code of q, 302 with half of P V: no one of them is the limit.  32 chains of 16
// rows take 95, 257 nodes over 8192 slots 65: beginnings and ends of tiles.  Slower were a thread to
// a row with two jobs of 64 keys in flight and four converting warps (381 for the chunk, 98 for the
// chains), the same with K turned into fp16 too, so that all MMAs are of a kind (381, 103), and
// halves that take turns with scores of 64 keys of their own, m and r handed on without a
// barrier (351, 108: MMAs 64 keys wide read q twice as often).
constexpr int kStepT = 128;
// Registers with NG = 2: the launch's 96 for each of five warpgroups, of which the four of
// the softmax take 104 and the other one keeps 64.  The compiler plans for 96 and spills 394
// bytes (572 read back) in a kernel; NG = 1, with 128, spills none.
constexpr int kRegsSoftmax = 104, kRegsOther = 64;
static_assert(4 * kRegsSoftmax + kRegsOther <= 5 * 96, "register split");

template <int HD, int NG>
struct Tc {
  static constexpr int kGroup = NG == 2 ? 128 : 64;         // rows of a softmax group, two threads to a row
  static constexpr int kRows = kGroup * NG, kWarps = kRows / 16;
  static constexpr int kThreads = NG == 2 ? 640 : 256, kPerSm = NG == 2 ? 1 : 2;
  // Warps.  A warp reaches the TMEM lanes (rows) of its number modulo 4 alone.
  static constexpr int kLoad = NG == 2 ? 16 : 2, kIssue = kLoad + 1, kConvert = NG == 2 ? 18 : 6, kConv = 2;
  using Geo = PagedGeo<kRows, kStepT, NG == 2 ? 12 : 3, 128, NG == 2 ? 1 : 3>;
  static constexpr int kAtomQ = kGroup * 128;               // 128 bytes of a group's rows of Q
  static constexpr int kTileQ = (HD / 64) * kAtomQ;         // hi and lo
  static constexpr int kKeys = NG == 2 ? 128 : 64;          // of a ring slot
  static constexpr int kPer = kStepT / kKeys;               // slots of a step's K, or V
  static constexpr int kSlot = kKeys * HD;                  // of codes
  static constexpr int kAtom = kKeys * 128, kTileV = (HD / 64) * kAtom;     // of values in fp16
  static constexpr int kK = NG == 2 ? 3 : 4, kV = NG == 2 ? 2 : 3, kC = 2;  // ring slots
  static constexpr int kRingK = NG * kTileQ, kRingV = kRingK + kK * kSlot, kRingC = kRingV + kV * kSlot;
  static constexpr int kBar = kRingC + kC * kTileV;
  static constexpr int kBars = 2 * (kK + kV + kC) + 10;
  static constexpr int kWait = kBar + kBars * 8, kWord = kWait + kThreads / 32 * 8;
  static constexpr int kNote = kWord + 16, kScale = (kNote + 64 + 15) / 16 * 16, kMl = kScale + 8 * 64;
  static constexpr int kSwap = kMl + (NG == 2 ? 1024 : 0);
  static constexpr int kBytes = kSwap + NG * 2 * kGroup * 4;
  static constexpr int kTmem = 256 * NG;                    // S_x at 128 x (P_x over it), then O_x
  static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "shared memory of an SM");
};

struct TcMaps {
  CUtensorMap k, v;    // pools as rows of head_dim bytes, box min(page_size, slot) rows
};

template <int HD, int NG>
__global__ void __launch_bounds__(Tc<HD, NG>::kThreads, Tc<HD, NG>::kPerSm)
paged_attn_tc_e4m3_kernel(const __grid_constant__ TcMaps maps, const PagedE4M3Params p) {
  using S = Tc<HD, NG>;
  using Geo = typename S::Geo;
  constexpr int kPer = S::kPer, GT = S::kGroup;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (ptx::smem_addr(smem) & 1023) {                         // (the swizzle counts on it)
    record_status(p.status, DFLASH_ERR_UNSUPPORTED);
    return;
  }
  uint8_t* sQ = smem;                                        // [NG][HD / 64][GT][128]
  uint8_t* sK = smem + S::kRingK;                            // slots of [kKeys][HD] codes
  uint8_t* sV = smem + S::kRingV;
  uint8_t* sC = smem + S::kRingC;                            // slots of [HD / 64][kKeys][64] fp16
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint64_t *k_full = bar, *k_empty = k_full + S::kK, *v_full = k_empty + S::kK, *v_empty = v_full + S::kV;
  uint64_t *c_full = v_empty + S::kV, *c_empty = c_full + S::kC;
  uint64_t* q_full = c_empty + S::kC;
  uint64_t* s_ready = q_full + 1;                            // [2]
  uint64_t* p_ready = q_full + 3;                            // [2][half]
  uint64_t* pv_done = q_full + 7;                            // [2]
  uint64_t* drain = q_full + 9;
  uint64_t* wait_ns = reinterpret_cast<uint64_t*>(smem + S::kWait) + (threadIdx.x >> 5);   // limit of a wait
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::kWord);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  volatile int* s_last = reinterpret_cast<volatile int*>(tslot + 2);    // [2]
  // keys with a NaN: [step % 4][16 keys], steps counted over all pieces.  A group reads a step's when it has its next
  // scores, before it hands out P for them; the converting warps are two steps past that
  // at most.
  volatile uint16_t* notes = reinterpret_cast<volatile uint16_t*>(smem + S::kNote);
  // (2^a, b) of a step's blocks: [step % 8][8].  The loads are at most the K ring's three
  // steps past the scores, those two past the softmax.
  float2* sScale = reinterpret_cast<float2*>(smem + S::kScale);
  float2* sMl = reinterpret_cast<float2*>(smem + S::kMl);    // [128] (NG = 2)
  // what a row's two threads tell each other: [half][NG][GT]
  volatile float* sSwap = reinterpret_cast<volatile float*>(smem + S::kSwap);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kLoad = S::kLoad, kIssue = S::kIssue, kConvert = S::kConvert;
  if (tid == 0) {
    for (int s = 0; s < S::kK; ++s) {
      ptx::mbar_init(&k_full[s], 1);
      ptx::mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < S::kV; ++s) {
      ptx::mbar_init(&v_full[s], 1);
      ptx::mbar_init(&v_empty[s], S::kConv);
    }
    for (int s = 0; s < S::kC; ++s) {
      ptx::mbar_init(&c_full[s], S::kConv);
      ptx::mbar_init(&c_empty[s], 1);
    }
    ptx::mbar_init(q_full, S::kWarps);
    for (int x = 0; x < 2; ++x) {
      ptx::mbar_init(&s_ready[x], 1);
      ptx::mbar_init(&p_ready[2 * x], GT / 32);
      ptx::mbar_init(&p_ready[2 * x + 1], GT / 32);
      ptx::mbar_init(&pv_done[x], 1);
    }
    ptx::mbar_init(drain, 1);
    *abort = 0;
    ptx::fence_mbar_init();
  }
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
  auto wait = [&](uint64_t* b, uint32_t parity) {            // bounded
    if (ptx::mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!ptx::mbar_try_wait(b, parity))
      if (*abort || global_ns() - t0 > *wait_ns) return false;
    return true;
  };
  auto all = [&](bool landed) { return __all_sync(0xffffffffu, landed); };

  // ---------------- values into fp16 ----------------
  auto convert = [&]() {
    constexpr int kPieces = HD / 16, kRound = 32 / kPieces, kMine = S::kKeys / S::kConv;
    const int w = warp - kConvert;
    const int ch = lane % kPieces, flip = HD == 128 ? ch >> 2 : 0;
    uint32_t iv = 0;                                         // slots converted
    bool ok = true;
    for (PagedPiece pc; c.left > 0 && ok; paged_next<Geo>(p, pc, &c)) {
      pc = PagedPiece::of<Geo>(c);
      if (pc.n <= 0) continue;
      const int kend = c.rq.key_end<Geo>(c.j, p.heads);
      const int plain = min(c.rq.masked ? c.rq.p0 : c.rq.p0 + p.heads.quot(c.j * S::kRows) + 1, kend);
      for (int i = 0; i < pc.n && ok; ++i) {
        const int key0 = (pc.first + i) * kStepT;
        const bool check = key0 + kStepT > plain;
        for (int part = 0; part < kPer && ok; ++part, ++iv) {
          const uint32_t s = iv % S::kV, t = iv % S::kC;
          ok = all(wait(&v_full[s], iv / S::kV & 1u) && wait(&c_empty[t], (iv / S::kC & 1u) ^ 1u));
          if (!ok) break;
          const uint8_t* from = sV + s * S::kSlot;
          uint8_t* to = sC + t * S::kTileV;
          auto take = [&](int k0) {
            const int key = w * kMine + k0 + lane / kPieces;
            return *reinterpret_cast<const uint4*>(
                from + key * HD + ((HD == 128 ? ch ^ (key & 7) : ch ^ ((key >> 1) & 3)) << 4));
          };
          auto put = [&](int k0, const uint4& u) {
            const int key = w * kMine + k0 + lane / kPieces;
            const uint4 a = make_uint4(half2_lo(u.x), half2_hi(u.x), half2_lo(u.y), half2_hi(u.y));
            const uint4 b = make_uint4(half2_lo(u.z), half2_hi(u.z), half2_lo(u.w), half2_hi(u.w));
            // 32 bytes of the row's 64-column atom; the upper half's lanes store the other
            // piece first (no bank conflicts)
            uint8_t* row = to + (ch >> 2) * S::kAtom + key * 128;
            const int c16 = (ch & 3) * 2;
            *reinterpret_cast<uint4*>(row + (((c16 + flip) ^ (key & 7)) << 4)) = flip ? b : a;
            *reinterpret_cast<uint4*>(row + (((c16 + 1 - flip) ^ (key & 7)) << 4)) = flip ? a : b;
          };
          if (!check) {
#pragma unroll 1
            for (int k0 = 0; k0 < kMine; k0 += 4 * kRound) {
              uint4 u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) u[k] = take(k0 + k * kRound);
#pragma unroll
              for (int k = 0; k < 4; ++k) put(k0 + k * kRound, u[k]);
            }
          } else {
            uint32_t bad = 0;                                // of 16 keys
#pragma unroll 1
            for (int k0 = 0; k0 < kMine; k0 += kRound) {
              uint4 u = take(k0);
              if (key0 + part * S::kKeys + w * kMine + k0 + lane / kPieces >= kend) u = make_uint4(0, 0, 0, 0);
              const uint4 x = make_uint4(nan_bytes(u.x), nan_bytes(u.y), nan_bytes(u.z), nan_bytes(u.w));
              const uint32_t hit = __ballot_sync(0xffffffffu, (x.x | x.y | x.z | x.w) != 0);
              for (int k = 0; k < kRound; ++k)
                if ((hit >> (k * kPieces)) & ((1u << kPieces) - 1u)) bad |= 1u << ((k0 + k) & 15);
              put(k0, make_uint4(u.x & ~x.x, u.y & ~x.y, u.z & ~x.z, u.w & ~x.w));
              if (((k0 + kRound) & 15) == 0) {
                if (lane == 0)
                  notes[(iv / kPer & 3) * 8 + (part * S::kKeys + w * kMine + k0) / 16] = static_cast<uint16_t>(bad);
                bad = 0;
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&c_full[t]);
            ptx::mbar_arrive(&v_empty[s]);
          }
        }
      }
    }
    if (!ok && lane == 0) fail();
  };
  // ---------------- loads ----------------
  auto load = [&]() {
    const int box = min(1 << p.pv.page_shift, S::kKeys);
    const int nb = kStepT / box;                             // boxes of a step's K, or V
    const int per_slot = S::kKeys / box;
    const uint64_t pol = ptx::policy_evict_last();
    if (lane == 0) {
      ptx::prefetch_tmap(&maps.k);
      ptx::prefetch_tmap(&maps.v);
    }
    const int nowhere = (p.pv.n_pages * p.pv.n_kv) << p.pv.page_shift;   // past the pool: zeros
    uint32_t ik = 0, iv = 0;                                 // slots loaded
    bool ok = true;
    for (PagedPiece pc; c.left > 0 && ok; paged_next<Geo>(p, pc, &c)) {
      pc = PagedPiece::of<Geo>(c);
      if (pc.n <= 0) continue;
      const int n = pc.n, kend = c.rq.key_end<Geo>(c.j, p.heads);
      const int32_t* table = p.pv.table + (size_t)c.r * p.pv.table_ld;
      // this lane's 16 slots of step i (lanes 0 .. 7): their page's table entry, asked for
      // two steps ahead, and their place in the pool and scales, one step ahead
      auto entry_of = [&](int i) {
        const int t = (pc.first + i) * kStepT + lane * kScaleBlock;
        return lane < 8 && i < n && t < kend ? __ldg(table + (t >> p.pv.page_shift)) : -1;
      };
      bool missing = false;
      struct Place {
        int row;
        uint32_t a, b;
      };
      auto place_of = [&](int i, int page) {
        const int t = (pc.first + i) * kStepT + lane * kScaleBlock;
        Place at = {nowhere, 127u, 127u};
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.pv.n_pages)) {
          const long long row = pool_row(p.pv, page, c.g, t);
          at.row = static_cast<int>(row);
          at.a = __ldg(p.k_scale + row / kScaleBlock);
          at.b = __ldg(p.v_scale + row / kScaleBlock);
        } else {
          missing |= lane < 8 && i < n && t < kend;
        }
        return at;
      };
      int entry = entry_of(0);
      Place next = place_of(0, entry);
      entry = entry_of(1);
      for (int i = 0; i < n && ok; ++i) {
        const Place now = next;
        if (i + 1 < n) next = place_of(i + 1, entry);
        entry = entry_of(i + 2);
        // lane b's box: the first of its 16-slot blocks
        const int y = __shfl_sync(0xffffffffu, now.row, min(lane * box / kScaleBlock, 7));
        auto fill = [&](uint64_t* full, uint64_t* empty, uint32_t it, int slots, uint8_t* ring, const CUtensorMap* map,
                        int part) {
          const uint32_t s = it % slots;
          if (!all(wait(&empty[s], (it / slots & 1u) ^ 1u))) return false;
          if (lane == 0) ptx::mbar_arrive_expect_tx(&full[s], S::kSlot);
          __syncwarp();
          const int b = lane - part * per_slot;              // this lane's box in the slot
          if (b >= 0 && b < per_slot && lane < nb) ptx::tma_load_2d(ring + s * S::kSlot + b * box * HD, map, &full[s], 0, y, pol);
          return true;
        };
        for (int part = 0; part < kPer && ok; ++part, ++ik) {
          if (part == 0) {                                   // (the scales before the keys' arrival)
            const uint32_t s = ik % S::kK;
            ok = all(wait(&k_empty[s], (ik / S::kK & 1u) ^ 1u));
            if (!ok) break;
            if (lane < 8)
              sScale[(ik / kPer & 7) * 8 + lane] = make_float2(scale_of(now.a), exponent_of(now.b));
            __syncwarp();
          }
          ok = fill(k_full, k_empty, ik, S::kK, sK, &maps.k, part);
        }
        for (int part = 0; part < kPer && ok; ++part, ++iv)
          ok = fill(v_full, v_empty, iv, S::kV, sV, &maps.v, part);
      }
      // pages that are not there: an error if some row of the tile sees their slots
      if (__any_sync(0xffffffffu, missing))
        for (int t0 = pc.first * kStepT; t0 < min((pc.first + n) * kStepT, kend); t0 += box)
          if (page_of(p.pv, c.r, t0) < 0 && paged_seen<Geo>(p, c, t0, min(t0 + box, kend), lane) && lane == 0)
            record_status(p.status, DFLASH_ERR_INVALID_ARG);
    }
    if (!ok && lane == 0) fail();
    // every copy must land before the CTA exits
    auto landed = [&](uint64_t* full, uint32_t it, uint32_t slots) {
      for (uint32_t s = 0; s < slots && s < it; ++s)
        ptx::mbar_wait_bounded(&full[s], (it - 1 - s) / slots & 1u, kTimeoutNs, nullptr);
    };
    landed(k_full, ik, S::kK);
    landed(v_full, iv, S::kV);
  };
  // ---------------- MMA issue ----------------
  auto issue = [&]() {
    // The whole warp runs the loop, so that addresses and descriptors stay in
    // uniform registers; one elected lane issues.
    const bool elected = ptx::elect_one();
    const uint64_t dq = ptx::sw128_kmajor_desc(ptx::smem_addr(sQ));
    const uint64_t dk = HD == 128 ? ptx::sw128_kmajor_desc(ptx::smem_addr(sK)) : ptx::sw64_kmajor_desc(ptx::smem_addr(sK));
    const uint64_t dv = ptx::sw128_mnmajor_desc(ptx::smem_addr(sC), S::kAtom, 1024);
    constexpr uint32_t idesc_s = ptx::idesc_f32(128, S::kKeys);
    constexpr uint32_t idesc_pv = ptx::idesc_f32(128, HD) | (1u << 16);   // B transposed
    uint32_t it = 0, unit = 0, np[2] = {0, 0};               // ring base, units, PV products of x
    uint32_t ks[kPer] = {}, vs[kPer] = {};                   // ring slots in use
    bool ok = true;
    for (PagedPiece pc; c.left > 0 && ok; paged_next<Geo>(p, pc, &c)) {
      pc = PagedPiece::of<Geo>(c);
      if (pc.n <= 0) continue;
      const int n = pc.n, nt = NG == 2 && min(c.rq.n * p.heads.G - c.j * S::kRows, S::kRows) > 128 ? 2 : 1;
      ok = all(wait(q_full, unit & 1u));
      const int jobs0 = NG == 1 || nt == 2 ? n : (n + 1) / 2, jobs1 = NG == 1 ? 0 : (nt == 2 ? n : n / 2);
      // group x's i-th job is this step; ring slots of a step are numbered on from `it`
      auto step_of = [&](int x, int i) { return NG == 1 || nt == 2 ? i : 2 * i + x; };
      auto slot_at = [&](uint32_t at, int slots) { return __shfl_sync(0xffffffffu, at % slots, 0); };
      // Waits that the loads decide come before the one that the softmax decides, and
      // between that one and the next scores there is nothing but MMAs.
      auto scores = [&](int x) {                             // one lane: S_x of the K in ks
        const uint64_t q0 = dq + (nt == 2 ? x * (S::kTileQ >> 4) : 0);
#pragma unroll
        for (int part = 0; part < kPer; ++part) {
          const uint32_t s = ks[part];
          const uint64_t k0 = dk + s * (S::kSlot >> 4);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {             // hi, then lo
            const int lo = kk / (HD / 32), at = kk % (HD / 32) * 32;
            ptx::mma_e4m3(tbase + 128 * x + part * S::kKeys,
                          q0 + ((lo * (HD == 128 ? S::kAtomQ : 64) + at) >> 4), k0 + (at >> 4), idesc_s,
                          kk > 0 ? 1u : 0u);
          }
          if (part == kPer - 1) ptx::mma_commit(&s_ready[x]);
          if (nt == 1 || x == 1) ptx::mma_commit(&k_empty[s]);
        }
      };
      auto wait_k = [&](int x, int i) {
        const uint32_t at = it + kPer * step_of(x, i);
        bool got = true;
#pragma unroll
        for (int part = 0; part < kPer; ++part) {
          ks[part] = slot_at(at + part, S::kK);
          got = got && all(wait(&k_full[(at + part) % S::kK], (at + part) / S::kK & 1u));
        }
        return got;
      };
      // job i of group x: P V, then the scores of job i + 1
      auto turn = [&](int x, int i, bool more) {
        const bool shared = nt == 2 && x == 1;               // group 0 has waited for these
        const uint32_t at = it + kPer * step_of(x, i);
        if (!shared) {
#pragma unroll
          for (int part = 0; part < kPer; ++part) {
            vs[part] = slot_at(at + part, S::kC);
            if (!all(wait(&c_full[(at + part) % S::kC], (at + part) / S::kC & 1u))) return false;
          }
          if (more && !wait_k(x, i + 1)) return false;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {                        // P arrives in two halves
          if (!all(wait(&p_ready[2 * x + h], np[x] & 1u))) return false;
          ptx::tc_fence_after();
          if (elected) {
            const uint32_t s = vs[kPer == 2 ? h : 0];
            const uint64_t v0 = dv + s * (S::kTileV >> 4);
#pragma unroll
            for (int j = 4 * h; j < 4 * h + 4; ++j)
              ptx::mma_bf16_ta(tbase_o + 128 * x, tbase + 128 * x + 64 * h + 8 * (j & 3),
                               v0 + (j % (S::kKeys / 16)) * (2048 >> 4), idesc_pv, (i > 0 || j > 0) ? 1u : 0u);
            if (h == 1) ptx::mma_commit(&pv_done[x]);
            if ((kPer == 2 || h == 1) && (nt == 1 || x == 1)) ptx::mma_commit(&c_empty[s]);
            if (h == 1 && more) scores(x);
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
        if (ok && elected) scores(x);
        __syncwarp();
      }
      for (int i = 0; i < jobs0 && ok; ++i) {
        ok = turn(0, i, i + 1 < jobs0);
        if (ok && i < jobs1) ok = turn(1, i, i + 1 < jobs1);
      }
      it += kPer * n;
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
  };
  // ---------------- softmax ----------------
  // Group x's rows, two threads to a row: half h takes 64 of a step's keys, and half of
  // O's columns.  Both know m and r; each has a sum of its own.
  auto softmax = [&]() {
    constexpr int kCols = HD / 2;
    const int x = NG == 2 ? (warp >> 2) & 1 : 0, h = NG == 2 ? warp >> 3 : warp >> 2;
    const int wg = NG == 2 ? warp & 3 : warp & 1, row = wg * 32 + lane;
    const int pair = 1 + x * 4 + wg, group = 9 + x, everyone = 11;       // barriers
    const uint32_t lane_off = static_cast<uint32_t>(wg * 32) << 16;
    const uint32_t aS = tbase + 128 * x + lane_off, aO = tbase_o + 128 * x + kCols * h + lane_off;
    volatile float *said = sSwap + (h * NG + x) * GT + row, *heard = sSwap + ((h ^ 1) * NG + x) * GT + row;
    auto swap = [&](float v) {                               // the other thread's value
      *said = v;
      ptx::named_bar_sync(pair, 64);
      const float o = *heard;
      ptx::named_bar_sync(pair, 64);
      return o;
    };
    uint32_t it = 0, nj = 0;                                 // steps, jobs of this group
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
      const bool dead = rho0 + wg * 32 >= nG;        // no live row in this warp
      // Q as two codes into shared memory (rows of 128 bytes, 128-byte swizzle), half a row
      // to a thread.  count: what a score of the codes counts
      float count = 0.f;
      if (!dead) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(rq.row0 + tok) * p.q_ld +
                                                          (long long)head * HD + kCols * h);
        uint4 u[kCols / 8];
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) u[i] = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
        }
        top = max(top, __float_as_uint(swap(__uint_as_float(top))));
        const int e = max(static_cast<int>(top >> 7), 16);                               // biased exponent
        const float up = __uint_as_float(static_cast<uint32_t>(261 - e) << 23);          // 2^(134 - e)
        count = __uint_as_float(static_cast<uint32_t>(e - 7) << 23) * p.scale_log2;
        if (nt == 2 || x == 0) {
          uint8_t* tile = sQ + (nt == 2 ? x : 0) * S::kTileQ + row * 128;
#pragma unroll
          for (int i = 0; i < kCols / 8; i += 2) {           // 16 elements: a piece of hi, one of lo
            uint32_t hi[4] = {}, lo[4] = {};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint4& q = u[i + (k >> 2)];
              const uint32_t w = (k & 3) == 0 ? q.x : (k & 3) == 1 ? q.y : (k & 3) == 2 ? q.z : q.w;
              float2 v = make_float2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
              v.x = fmaf(v.x, 0.f, v.x);                     // (an infinity becomes NaN)
              v.y = fmaf(v.y, 0.f, v.y);
              const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
              const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(a, __NV_E4M3)));
              const __nv_fp8x2_storage_t b =
                  __nv_cvt_float2_to_fp8x2(make_float2(v.x - f.x, v.y - f.y), __NV_SATFINITE, __NV_E4M3);
              hi[k >> 1] |= static_cast<uint32_t>(a) << (16 * (k & 1));
              lo[k >> 1] |= static_cast<uint32_t>(b) << (16 * (k & 1));
            }
            auto put = [&](int byte, const uint32_t (&w)[4]) {           // byte of the row: atom, piece
              *reinterpret_cast<uint4*>(tile + (byte >> 7) * S::kAtomQ + ((((byte & 127) >> 4) ^ (row & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            };
            put(kCols * h + 8 * i, hi);
            put(HD + kCols * h + 8 * i, lo);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(q_full);

      // first slot past what the row sees (causal), the mask row, and the keys
      // that every row of the warp, and of the whole tile, sees
      const int lim = live ? (rq.masked ? kend : min(rq.p0 + tok + 1, kend)) : 0;
      const uint32_t* mrow = rq.masked ? p.mask + (size_t)(rq.row0 + tok) * p.mask_ld : nullptr;
      const int first = p.heads.quot(min(rho0 + wg * 32, nG - 1));
      const int plain_w = dead ? 0 : min(rq.masked ? rq.p0 : rq.p0 + first + 1, kend);
      const int plain_t = min(rq.masked ? rq.p0 : rq.p0 + p.heads.quot(tile0) + 1, kend);
      auto sees = [&](int k) {                               // keys [k, k + 32), a bit to a key
        uint32_t bits = low_bits(lim - k);
        if (rq.masked && bits) bits &= seen_word(mrow, p.mask_ld, k - rq.p0);
        return bits;
      };
      float m = -CUDART_INF_F, r = -CUDART_INF_F, l = 0.f;
      // A step's P V ran with zeros for NaN codes.  Once it is done (the next scores are, or
      // pv_done), a row that sees such a key becomes NaN in the code's column.
      int late = -1;                                         // first key of the step to be looked through, or none
      uint32_t late_note = 0;
      auto repair = [&]() {
        if (late < 0 || dead) return;
#pragma unroll 1
        for (int g = 0; g < 8; ++g) {
          uint32_t keys = notes[late_note * 8 + g];
          if (keys == 0) continue;                           // (warp-uniform)
          const uint32_t mine = sees(late + 16 * g);
          while (keys) {
            const int j = __ffs(keys) - 1;
            keys &= keys - 1;
            const int key = late + 16 * g + j, page = page_of(p.pv, c.r, key);
            if (page < 0) continue;
            const uint8_t* v = static_cast<const uint8_t*>(p.pv.v) + pool_row(p.pv, page, c.g, key) * HD + kCols * h;
            const bool see = (mine >> j) & 1u;
#pragma unroll 1
            for (int cb = 0; cb < kCols / 16; ++cb) {
              float o[16];
              ptx::tmem_ld_32x16(aO + 16 * cb, o);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (see && (v[16 * cb + e] & 127) == 127) o[e] = CUDART_NAN_F;
              ptx::tmem_st_32x16(aO + 16 * cb, o);
              ptx::tmem_wait_st();
            }
          }
        }
      };
      // (after a wait has run out the loop only runs on to everyone's barrier)
      for (int i = 0; i < jobs; ++i, ++nj) {
        if (!ok) continue;
        const int t = NG == 1 || nt == 2 ? i : 2 * i + x, key0 = (pc.first + t) * kStepT;
        ok = all(wait(&s_ready[x], nj & 1u));
        if (dead) {
          if (ok && lane == 0) ptx::mbar_arrive(&p_ready[2 * x + h]);
          continue;
        }
        ptx::tc_fence_after();
        if (ok && late >= 0) repair();
        late = key0 + kStepT > plain_t ? key0 : -1;
        late_note = it + t & 3;
        const float2* scale = sScale + (it + t & 7) * 8 + 4 * h;
        // a block's factor (no infinity times zero, nor zero times infinity)
        auto factor = [&](float a) { return fminf(fmaxf(count * a, 0x1p-126f), 0x1p90f); };
        uint32_t u[2][32];
        ptx::tmem_ld_32x32(aS + 64 * h, u[0]);
        ptx::tmem_ld_32x32(aS + 64 * h + 32, u[1]);
        const int k0 = key0 + 64 * h;
        uint32_t seen[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        const bool hide = k0 + 64 > plain_w;                 // some key is hidden from some row
        if (hide) {
          seen[0] = sees(k0);
          seen[1] = sees(k0 + 32);
        }
        ptx::tmem_wait_ld();
        if (hide) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((seen[b] >> j) & 1u)) u[b][j] = 0xff800000u;
        }
        float top[4], mx = -CUDART_INF_F, mr = -CUDART_INF_F;       // of a block; of all; with its exponent
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t* w = &u[g >> 1][16 * (g & 1)];
          float a0 = fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])), __uint_as_float(w[2]));
          float a1 = fmaxf(fmaxf(__uint_as_float(w[3]), __uint_as_float(w[4])), __uint_as_float(w[5]));
#pragma unroll
          for (int j = 6; j < 14; j += 4) {
            a0 = fmaxf(fmaxf(a0, __uint_as_float(w[j])), __uint_as_float(w[j + 1]));
            a1 = fmaxf(fmaxf(a1, __uint_as_float(w[j + 2])), __uint_as_float(w[j + 3]));
          }
          a0 = fmaxf(fmaxf(a0, __uint_as_float(w[14])), __uint_as_float(w[15]));
          const float2 sc = scale[g];
          top[g] = fmaxf(a0, a1) * factor(sc.x);
          mx = fmaxf(mx, top[g]);
          mr = fmaxf(mr, (top[g] - m) + sc.y);               // (NaN where nothing has been seen)
        }
        const bool raise = mx > m + kLag || mr > r + kLag;
        if (ptx::named_bar_or(pair, 64, raise || !ok)) {     // (rare)
          const float other = swap(ok ? mx : CUDART_NAN_F);
          ok = all(ok && !(other != other));
          if (!ok) continue;
          const float base = fmaxf(m, fmaxf(mx, other));
          mr = -CUDART_INF_F;
#pragma unroll
          for (int g = 0; g < 4; ++g) mr = fmaxf(mr, (top[g] - base) + scale[g].y);
          mr = fmaxf(mr, swap(mr));
          float f = 1.f;
          if (base > m + kLag || mr > r + (m - base) + kLag) {
            const float was = m - base + r, r2 = fmaxf(was, mr);
            f = ex2(was - r2);
            l *= ex2(m - base);
            m = base;
            r = r2;
          }
          if (i > 0) {
            // the products so far must be in O before it is scaled
            ok = all(wait(&pv_done[x], (nj - 1) & 1u));
            if (ok) {
              ptx::tc_fence_after();
#pragma unroll 1
              for (int b = 0; b < kCols / 16; ++b) {
                float o[16];
                ptx::tmem_ld_32x16(aO + 16 * b, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= f;
                ptx::tmem_st_32x16(aO + 16 * b, o);
              }
              ptx::tmem_wait_st();
            }
            ptx::tc_fence_before();
            if (ptx::named_bar_or(pair, 64, !ok)) ok = false;       // (P of either half meets all of O)
            if (!ok) continue;
          }
        }
        ptx::tc_fence_after();
        const bool none = m == -CUDART_INF_F;
        // Scores so large that d - m below would lose bits: s - m first, on its own (rare).
        const bool far = __any_sync(0xffffffffu, !none && fabsf(m) > 0x1p20f);
        if (far) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float f = factor(scale[g].x);
#pragma unroll
            for (int j = 16 * (g & 1); j < 16 * (g & 1) + 16; ++j)
              u[g >> 1][j] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(u[g >> 1][j]), f), none ? 0.f : m));
          }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {                        // P over the half's own scores
          const float2 sc = scale[g];
          // 2^-60 of the largest weight is as good as none: l keeps its share
          const float d = none ? 0.f : fmaxf(sc.y - r, -60.f), add = none || far ? d : d - m;
          const float f1 = far ? 1.f : factor(sc.x);
          const float2 f2 = make_float2(f1, f1), a2 = make_float2(add, add);
          float2 rs = make_float2(0.f, 0.f);
          uint32_t pk[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(u[g >> 1][16 * (g & 1) + 2 * j]),
                                                    __uint_as_float(u[g >> 1][16 * (g & 1) + 2 * j + 1])), f2, a2);
            const float2 w = make_float2(ex2(y.x), ex2(y.y));
            rs = __fadd2_rn(rs, w);
            pk[j] = pack_f16(w.x, w.y);
          }
          l = fmaf(rs.x + rs.y, ex2(-d), l);
          ptx::tmem_st_32x8(aS + 64 * h + 8 * g, pk);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&p_ready[2 * x + h]);
      }
      if (ok && jobs > 0) {
        ok = all(wait(&pv_done[x], (nj - 1) & 1u));
        if (ok) ptx::tc_fence_after();
        if (ok) repair();
      }
      if (ptx::named_bar_or(everyone, 2 * GT * NG, !ok)) {
        ok = false;
        break;
      }
      // ---- the tile's rows ----  (O with m as its reference: times 2^r)
      if (!dead) l += swap(l);
      // A weight may vanish beside another; NaN times it stays NaN.  Only what saw no key
      // counts for nothing.
      const bool some = m != -CUDART_INF_F;
      const float own = some ? ex2_low(r) : 0.f;
      float M = m, L = l, fa = own, fb = 0.f;                // weights of the two groups' halves
      bool both = false;                                     // the other group's half counts
      float* sB = reinterpret_cast<float*>(sQ);              // [128][HD], chunks of 4 swizzled
      if (NG == 2 && nt == 1) {
        if (x == 1 && !dead) {
          if (h == 0) sMl[row] = make_float2(m, l);
          if (jobs > 0) {
#pragma unroll
            for (int b = 0; b < kCols / 32; ++b) {
              uint32_t o[32];
              ptx::tmem_ld_32x32(aO + 32 * b, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4*>(sB + row * HD + 4 * ((kCols / 4 * h + 8 * b + j) ^ (row & 7))) =
                    make_float4(__uint_as_float(o[4 * j]) * own, __uint_as_float(o[4 * j + 1]) * own,
                                __uint_as_float(o[4 * j + 2]) * own, __uint_as_float(o[4 * j + 3]) * own);
            }
          }
        }
        ptx::named_bar_sync(everyone, 2 * GT * NG);
        if (x == 0 && !dead) {
          const float2 ml = sMl[row];
          both = ml.y != 0.f;
          if (both) {
            M = fmaxf(m, ml.x);
            const float f = l != 0.f ? ex2(m - M) : 0.f;
            fa = f * own;
            fb = ex2(ml.x - M);
            L = f * l + fb * ml.y;
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
      // The warp's 32 half rows in bf16 go out through shared memory, so that neighbouring
      // lanes write a row together: in a part of Q of its own, or, a lane each, in its
      // half of its row of the joined group, over columns that it has read.
      constexpr int kOut = HD / 16;                          // 16-byte pieces of a half row
      const bool joined = NG == 2 && nt == 1;
      const int stage_ld = joined ? HD * 4 : kCols * 2;
      uint8_t* stage = joined ? sQ + wg * 32 * stage_ld + h * kCols * 4 : sQ + ((h * NG + x) * (GT / 32) + wg) * 32 * stage_ld;
      auto put = [&](int b, const float (&o)[32], float inv) {    // 32 columns of the half row
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t w4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w4[e] = L == 0.f ? 0u : mmas::pack_bf16(o[8 * j + 2 * e] * inv, o[8 * j + 2 * e + 1] * inv);
          *reinterpret_cast<uint4*>(stage + lane * stage_ld + (((4 * b + j) ^ (lane & (kOut - 1))) << 4)) =
              make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
      };
      auto send = [&]() {
        __syncwarp();
        const unsigned long long mine_to = reinterpret_cast<unsigned long long>(
            p.out + (long long)(rq.row0 + tok) * p.out_ld + (long long)head * HD + kCols * h);
        const unsigned on = __ballot_sync(0xffffffffu, live);
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 32 / kOut) {
          const int rr = r0 + lane / kOut, ch = lane % kOut;
          uint4* to = reinterpret_cast<uint4*>(__shfl_sync(0xffffffffu, mine_to, rr)) + ch;
          const uint4 w = *reinterpret_cast<const uint4*>(stage + rr * stage_ld + ((ch ^ (rr & (kOut - 1))) << 4));
          if ((on >> rr) & 1u) *to = w;
        }
      };
      if (mine && !dead) {
        const float inv = 1.f / L;
#pragma unroll
        for (int b = 0; b < kCols / 32; ++b) {
          uint32_t u[32];
          ptx::tmem_ld_32x32(aO + 32 * b, u);
          ptx::tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = some ? __uint_as_float(u[j]) * fa : 0.f;
          if (both) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 v = *reinterpret_cast<const float4*>(sB + row * HD + 4 * ((kCols / 4 * h + 8 * b + j) ^ (row & 7)));
              o[4 * j] += fb * v.x;
              o[4 * j + 1] += fb * v.y;
              o[4 * j + 2] += fb * v.z;
              o[4 * j + 3] += fb * v.w;
            }
          }
          if (whole) {
            put(b, o, inv);
          } else if (live) {
            float4* po = reinterpret_cast<float4*>(p.part_o) + (slot * (HD / 4) + kCols / 4 * h + 8 * b) * GT + row;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              __stcg(po + j * GT, make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
          }
        }
        if (whole) send();
      }
      ptx::tc_fence_before();
      if (!whole && mine) {
        if (live && h == 0) __stcg(p.part_ml + slot * GT + row, make_float2(M, L));
        if (p.cut) {
          if (tid == 0 && c0 == static_cast<int>(blockIdx.x))   // its first piece
            p.cut[c0] = {c1, rq.row0, tile0, nG, c.g * p.heads.G};
        } else {
          __threadfence();
          ptx::named_bar_sync(group, 2 * GT);
          if (row == 0 && h == 0) s_last[x] = atomicAdd(p.arrive + NG * c0 + x, 1) == c1 - c0;
          ptx::named_bar_sync(group, 2 * GT);
          if (s_last[x]) {
            __threadfence();
            if (row == 0 && h == 0) p.arrive[NG * c0 + x] = 0;  // for the next call
            if (!dead) {
              M = -CUDART_INF_F;
#pragma unroll 4
              for (int cc = c0; cc <= c1; ++cc) M = fmaxf(M, __ldcg(p.part_ml + part_of(cc) * GT + row).x);
#pragma unroll 1
              for (int b = 0; b < kCols / 32; ++b) {
                float o[32] = {};
                L = 0.f;
                float2 ml = __ldcg(p.part_ml + part_of(c0) * GT + row);
                for (int cc = c0; cc <= c1; ++cc) {
                  const float2 now = ml;
                  if (cc < c1) ml = __ldcg(p.part_ml + part_of(cc + 1) * GT + row);
                  const float f = now.y != 0.f ? ex2(now.x - M) : 0.f;
                  L += f * now.y;
                  const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                                      (part_of(cc) * (HD / 4) + kCols / 4 * h + 8 * b) * GT + row;
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const float4 v = __ldcg(src + j * GT);
                    if (now.y != 0.f) {
                      o[4 * j] += f * v.x;
                      o[4 * j + 1] += f * v.y;
                      o[4 * j + 2] += f * v.z;
                      o[4 * j + 3] += f * v.w;
                    }
                  }
                }
                put(b, o, 1.f / L);
              }
              send();
            }
          }
        }
      }
      it += n;
      // the rows on their way out lie where the next tile's queries go
      ptx::named_bar_sync(everyone, 2 * GT * NG);
    }
    if (!ok) fail();
  };

  // (a warpgroup changes its registers in one instruction)
  if constexpr (NG == 2) {
    if (warp >= kLoad) {
      ptx::regs_dec<kRegsOther>();
      if (warp == kLoad) load();
      else if (warp == kIssue) issue();
      else convert();
    } else {
      ptx::regs_inc<kRegsSoftmax>();
      softmax();
    }
  } else {
    if (warp == kLoad) load();
    else if (warp == kIssue) issue();
    else if (warp >= kConvert) convert();
    else softmax();
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kIssue) {
    __syncwarp();
    ptx::tmem_dealloc(tbase, S::kTmem);
  }
}

template <int HD, int NG>
dflash_status launch_tc(PagedE4M3Params p, const dflash_pages_e4m3& pages, cudaStream_t st) {
  using S = Tc<HD, NG>;
  static_assert(S::kPerSm * NG <= kMostCtas && S::kPerSm * S::kRows <= 256, "the workspace's counters and slots");
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(paged_attn_tc_e4m3_kernel<HD, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  TcMaps maps;
  const int rows = pages.n_pages * pages.n_kv * pages.page_size;
  const int box = pages.page_size < S::kKeys ? pages.page_size : S::kKeys;
  if (!encode_bytes_map(&maps.k, pages.k, rows, HD, box) || !encode_bytes_map(&maps.v, pages.v, rows, HD, box))
    return set_error(DFLASH_ERR_CUDA, "paged attention e4m3: cannot encode the TMA descriptors");
  const int grid = num_sms() * S::kPerSm;
  // A few parts to a tile are joined by the last CTA to arrive, many by a kernel of their
  // own: the rule of the 16-bit cache (paged_attention.cu).
  const long long tiles = (p.n_rows * (long long)p.heads.G + S::kRows - 1) / S::kRows * p.pv.n_kv;
  if (tiles * 4 >= grid) p.cut = nullptr;
  {
    TraceScope ts("paged_attn_tc_e4m3", st);
    launch_k(paged_attn_tc_e4m3_kernel<HD, NG>, dim3(grid), dim3(S::kThreads), S::kBytes, st, maps, p);
  }
  if (p.cut) {
    TraceScope ts("paged_join", st);
    launch_k(paged_join_kernel<HD, NG, S::kGroup>, dim3(grid, S::kRows / 32), dim3(256), 0, st,
             static_cast<const PagedAttnParams&>(p));
  }
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
  if (num_sms() > kMostSms)
    return set_error(DFLASH_ERR_UNSUPPORTED, "paged attention e4m3: more than %d SMs", kMostSms);
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
  // The tile by the query rows of the largest request and KV head (8 KV heads of 128; tiles of
  // 8 / 16 / 64 / 256 rows, us):
  //   32 requests over 4096 slots:  8 rows 56 / 68 / 85 / 102, 16 rows 93 / 72 / 86 / 102,
  //     24 rows 133 / 123 / 88 / 103, 64 rows 323 / 228 / 87 / 104, 80 rows - / - / 152 / 120;
  //   1 request over 8192:  8 rows 21 / 24 / 29 / 29, 16 rows 21 / 28 / 29 / 29,
  //     32 rows 23 / 29 / 30 / 30, 64 rows 33 / 31 / 32 / 31, 128 rows - / - / 33 / 33.
  // Many slots take the smallest tile that holds the rows: theirs are read once.  Few are
  // joined from many parts, quickest where the rows are spread over several small tiles:
  //   16 rows: 1 x 2048 15 / 19 / 23 / -, 4 x 2048 19 / 22 / 25 / -, 2 x 16384 34 / 36 / 38 / -,
  //     4 x 16384 50 / 45 / 53 / -;
  //   32 rows: 4 x 2048 25 / 25 / 26 / -, 2 x 16384 50 / 44 / 38 / -.
  // The lengths are on the device; the page table's width bounds them.
  const long long rows = (long long)max_rows * p.heads.G;
  const bool few = (((long long)n_req * pages->n_kv * pages->table_ld) << p.pv.page_shift) <= 1 << 17;
  dflash_status e;
  if (rows <= (few ? 32 : 8))
    e = hd == 128 ? launch_small<128, 1>(p, *pages, st) : launch_small<64, 1>(p, *pages, st);
  else if (rows <= 16)
    e = hd == 128 ? launch_small<128, 2>(p, *pages, st) : launch_small<64, 2>(p, *pages, st);
  else if (rows <= Tc<128, 1>::kRows)
    e = hd == 128 ? launch_tc<128, 1>(p, *pages, st) : launch_tc<64, 1>(p, *pages, st);
  else
    e = hd == 128 ? launch_tc<128, 2>(p, *pages, st) : launch_tc<64, 2>(p, *pages, st);
  if (e) return e;
  return check_launch("paged attention e4m3");
}

}  // extern "C"
