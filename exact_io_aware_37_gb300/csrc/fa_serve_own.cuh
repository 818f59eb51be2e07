// The pass over the sequences' own cache rows of a decoding step
// (fa_decode_cache, fa_decode_shared).
//
// Mathematics.  For the rows of one (sequence b, key head h) -- its group * nq
// query rows, up to 16 WR of them a CTA -- S = Q K^T, P = 2^(c2 S - m),
// u += P V with a running maximum m and sum l.  Keys and values of the 8-bit
// cache enter the products as their codes (exact in fp16); the key's power of
// two multiplies its score, the value's power of two, 2^e, its weight: the
// weight that is rounded to fp16 is 2^(s + e - mu) with a running maximum mu of
// s + e of its own, so that the largest contribution, not the largest weight,
// sits at the top of fp16's range however unlike the rows' scales are.
//
// Bound.  Every cache row is read once: HBM.  A row of D codes costs 2 D
// multiply-adds for each of 16 padded query rows, which the warp-level MMA does
// in passing, so no tensor memory is used: with at most 64 rows an operand tile
// of 128 would be padding.
//
// Layout.  A CTA of 4 warps is WR row tiles x WK = 4 / WR key groups.  A key
// group streams stages of 4 KB of keys and 4 KB of values through a ring of
// its own: TMA writes them swizzled, so that both the 16-byte reads along a
// key (B operand of S) and those of four keys at one column block (B operand
// of P V) are free of bank conflicts; no block-wide barrier sits in the loop.
// Logical columns are permuted to make each lane's 16 bytes serve whole
// operands: keys through key_of, head-width elements through d_of.
//
// Schedule.  The tiles of all (sequence, head, row group) units are laid out in
// a row and cut into equal runs, one a CTA, from the lengths on the device;
// a unit that is cut leaves one state a run, joined by the merge kernel.
#pragma once

#include <math.h>

#include "fa_cache8.cuh"
#include "fa_internal.cuh"
#include "fa_serve.cuh"
#include "fa_tmap.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

constexpr int kOwnThreads = 128;

struct OwnParams {
  CUtensorMap tk, tv;
  ServeArgs a;
  int row_groups;
  bool q_f16;  // 8-bit cache: the queries' type (16-bit caches have the queries' type)
};

enum CacheKind { kE4m3, kBf16, kF16 };

template <int Kind, int D, int WR>
struct OwnCfg {
  static constexpr bool kCodes = Kind == kE4m3;
  static constexpr bool kMmaF16 = Kind != kBf16;
  static constexpr int kRowBytes = D * (kCodes ? 1 : 2);
  static constexpr int kPitch = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row in one swizzled block
  static constexpr int kBlocks = kRowBytes / kPitch;                // blocks side by side (D = 128 in 16 bits: 2)
  static constexpr int kHalf = 4096;                                // a stage's keys (or values)
  static constexpr int kKeys = own_stage_keys(kRowBytes);
  static constexpr int kBlockBytes = kKeys * kPitch;
  static constexpr int kWK = 4 / WR;
  static constexpr int kTile = kKeys * kWK;  // keys of a CTA's step
  static constexpr int kStages = 3 * WR;     // of a key group: 96 KB a CTA in all, two CTAs an SM
  static constexpr int kRing = kStages * 2 * kHalf;
  static constexpr int kSmem = kWK * kRing + 1024;
  static constexpr int kNT = kKeys / 8;   // 8-key tiles of a stage
  static constexpr int kKS = D / 16;      // 16-element steps of a score
  static constexpr int kDT = D / 8;       // 8-element tiles of an output row
  static constexpr int kRun = kRowBytes == 128 && kCodes ? 16 : 8;  // consecutive elements of a lane's output column
};

// Logical key n (0 .. 7) of an 8-key tile is row key_of(n): for 128-byte rows
// the two keys that one phase of a 16-byte read covers are four rows apart,
// which the swizzle sends to different banks.
template <int kPitch>
__device__ __forceinline__ int key_of(int n) {
  return kPitch == 128 ? (n >> 1) | ((n & 1) << 2) : n;
}
// The same for the 16-byte column block of logical column n.
__device__ __forceinline__ int block_of(int n) { return (n >> 1) | ((n & 1) << 2); }

// Byte offset of 16-byte chunk `chunk` of row `row` in a swizzled block.
template <int kPitch>
__device__ __forceinline__ int swz(int row, int chunk) {
  if constexpr (kPitch == 128)
    return row * 128 + ((chunk ^ (row & 7)) << 4);
  else
    return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// First element of the kRun consecutive ones of logical column n in output run
// `run` (the run holds 8-element tiles run * kRun .. + kRun - 1).
template <class C>
__device__ __forceinline__ int d_of(int n, int run) {
  if constexpr (C::kRun == 16) return block_of(n) * 16;
  if constexpr (C::kPitch == 64) return n * 8;
  return run * 64 + block_of(n) * 8;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// Elements of a word of values that are not finite become zero.
template <int Kind>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if constexpr (Kind == kE4m3) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (((w >> (8 * i)) & 0x7fu) == 0x7fu) w &= ~(0xffu << (8 * i));
  } else {
    constexpr uint32_t kExp = Kind == kBf16 ? 0x7f80u : 0x7c00u;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (((w >> (16 * i)) & kExp) == kExp) w &= ~(0xffffu << (16 * i));
  }
  return w;
}

template <int Kind, int D, int WR>
__global__ void __launch_bounds__(kOwnThreads, 2) own_kernel(const __grid_constant__ OwnParams p) {
  using C = OwnCfg<Kind, D, WR>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[C::kWK * C::kStages], bar_empty[C::kWK * C::kStages];
  __shared__ float s_m[C::kWK][16 * WR], s_l[C::kWK][16 * WR], s_mu[C::kWK][16 * WR];
  __shared__ OwnPlan plan;
  __shared__ int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const ServeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wk = warp / WR, wr = warp % WR;  // key group, row tile
  const int c = lane & 3, j = lane >> 2;
  const bool leader = wr == 0 && lane == 0;

  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kWK * C::kStages; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], WR);
    }
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
  }
  const int units = a.Hk * p.row_groups;  // of one sequence
  own_plan<kOwnThreads>(a, C::kTile, units, plan);  // ends with a block-wide barrier
  const WaitCtx w{&abort_flag, a.status, a.wait_limit_ns};

  const int rows = a.group * a.nq;
  uint8_t* ring = smem + wk * C::kRing;
  uint64_t* full = bar_full + wk * C::kStages;
  uint64_t* empty = bar_empty + wk * C::kStages;
  bool ok = true;
  unsigned issued = 0, taken = 0;  // stages of this key group so far

  long long t = plan.first;
  int b = plan.b;
  long long base = plan.base;  // tiles before sequence b
  while (t < plan.end) {
    const int len = seq_len(a, b);
    const int nt = own_tiles(len, C::kTile);
    if (t >= base + (long long)nt * units) {
      base += (long long)nt * units;
      ++b;
      continue;
    }
    // ---- the unit and the run of its tiles
    const int unit = (int)((t - base) / nt);
    const int tile0 = (int)((t - base) - (long long)unit * nt);
    const int tile1 = (int)min((long long)nt, tile0 + (plan.end - t));
    const int hk = unit / p.row_groups, row0 = (unit - hk * p.row_groups) * 16 * WR;
    const int slab = b * a.Hk + hk;
    const long long bh = slab;

    // stage i of this key group (i counts from tile0) holds keys k0(i) ..
    auto k0 = [&](int i) { return (tile0 + i) * C::kTile + wk * C::kKeys; };
    // stages with a key: all but perhaps the last
    const int n = max(0, min(tile1 - tile0, (len - wk * C::kKeys + C::kTile - 1) / C::kTile - tile0));
    auto load = [&](int i) {
      const unsigned s = issued % C::kStages;
      mbar_arrive_expect_tx(&full[s], 2 * C::kHalf);
      uint8_t* dst = ring + s * 2 * C::kHalf;
#pragma unroll
      for (int blk = 0; blk < C::kBlocks; ++blk) {
        tma_load_3d(dst + blk * C::kBlockBytes, &p.tk, &full[s], blk * 64, k0(i), slab);
        tma_load_3d(dst + C::kHalf + blk * C::kBlockBytes, &p.tv, &full[s], blk * 64, k0(i), slab);
      }
      ++issued;
    };
    int next = 0;  // stages of this run asked for
    // With several row tiles a stage is filled again once their warps are all done
    // with it; one stage of slack keeps the leader from waiting for the one just read.
    auto refill = [&] {
      while (leader && ok && next < n && issued - taken < C::kStages - (WR > 1 ? 1 : 0)) {
        if (WR > 1 && issued >= C::kStages &&
            !mbar_wait(&empty[issued % C::kStages], (issued / C::kStages - 1) & 1, w))
          ok = false;
        else
          load(next++);
      }
    };
    refill();

    // ---- query rows row0 + 16 wr + j and + 8, as A operands
    const int r_lo = row0 + 16 * wr + j, r_hi = r_lo + 8;
    uint32_t qa[C::kKS][4];
    float rs_lo = a.c2, rs_hi = a.c2;  // a row's factor from products to log2 units
    {
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + bh * rows * D;
#pragma unroll
      for (int ks = 0; ks < C::kKS; ++ks) {
        const int d0 = C::kCodes ? 16 * (c + 4 * (ks >> 2)) + 4 * (ks & 3) : 8 * (c + 4 * (ks >> 1)) + 4 * (ks & 1);
        const uint2 lo = r_lo < rows ? *reinterpret_cast<const uint2*>(q + (long long)r_lo * D + d0) : make_uint2(0, 0);
        const uint2 hi = r_hi < rows ? *reinterpret_cast<const uint2*>(q + (long long)r_hi * D + d0) : make_uint2(0, 0);
        qa[ks][0] = lo.x;
        qa[ks][1] = hi.x;
        qa[ks][2] = lo.y;
        qa[ks][3] = hi.y;
      }
      if constexpr (C::kCodes) {
        // The products run in fp16.  A row is scaled by the power of two that puts
        // its largest element between 2^14 and 2^15: exact for bf16 and fp16 down
        // to 2^-38 of that element, where fp16's subnormals end.
        auto value = [&](uint32_t h) {  // the element in the low 16 bits
          return p.q_f16 ? __half2float(__ushort_as_half((unsigned short)h)) : __uint_as_float(h << 16);
        };
        float big_lo = 0.f, big_hi = 0.f;
#pragma unroll
        for (int ks = 0; ks < C::kKS; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& big = (e & 1) ? big_hi : big_lo;
            big = fmaxf(big, fmaxf(fabsf(value(qa[ks][e] & 0xffffu)), fabsf(value(qa[ks][e] >> 16))));
          }
#pragma unroll
        for (int m = 1; m <= 2; m <<= 1) {
          big_lo = fmaxf(big_lo, __shfl_xor_sync(0xffffffffu, big_lo, m));
          big_hi = fmaxf(big_hi, __shfl_xor_sync(0xffffffffu, big_hi, m));
        }
        auto power = [](float big) {  // k with big 2^k in [2^14, 2^15), at most 126; 0 for what is not finite
          const int e = (int)(__float_as_uint(big) >> 23);
          return e == 255 ? 0 : min(141 - e, 126);
        };
        const int k_lo = power(big_lo), k_hi = power(big_hi);
        const float f_lo = __uint_as_float((uint32_t)(127 + k_lo) << 23);
        const float f_hi = __uint_as_float((uint32_t)(127 + k_hi) << 23);
#pragma unroll
        for (int ks = 0; ks < C::kKS; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = (e & 1) ? f_hi : f_lo;
            qa[ks][e] = pack_f16x2(value(qa[ks][e] & 0xffffu) * f, value(qa[ks][e] >> 16) * f);
          }
        rs_lo *= __uint_as_float((uint32_t)(127 - k_lo) << 23);
        rs_hi *= __uint_as_float((uint32_t)(127 - k_hi) << 23);
      }
    }
    // keys visible to the two rows, and to every row
    const int lim_lo = a.causal ? min(len, max(0, len - a.nq + r_lo % a.nq + 1)) : len;
    const int lim_hi = a.causal ? min(len, max(0, len - a.nq + r_hi % a.nq + 1)) : len;
    const int lim_all = a.causal ? max(0, len - a.nq + 1) : len;

    float acc[C::kDT][4];
#pragma unroll
    for (int d = 0; d < C::kDT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[d][e] = 0.f;
    // running maxima (log2 units) of the scores and, with codes, of score + value
    // exponent; this lane's share of the sums
    float m_lo = -INFINITY, m_hi = -INFINITY, mu_lo = -INFINITY, mu_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;

    // the exponents of a stage's keys: lane x holds those of keys x and x + 32
    auto load_exps = [&](int i) -> uint32_t {
      uint32_t e = 0;
      if constexpr (C::kCodes) {
#pragma unroll
        for (int h = 0; h < C::kKeys / 32; ++h) {
          const int key = k0(i) + 32 * h + lane;
          if (i < n && key < len) {
            const long long at = bh * a.cap + key;
            e |= ((uint32_t)__ldg(a.k_exp + at) | (uint32_t)__ldg(a.v_exp + at) << 8) << (16 * h);
          }
        }
      }
      return e;
    };
    uint32_t exps = load_exps(0);

    for (int i = 0; i < n && ok; ++i) {
      const unsigned s = taken % C::kStages;
      const uint32_t exps_now = exps;
      exps = load_exps(i + 1);  // a stage ahead
      if (!warp_wait(&full[s], (taken / C::kStages) & 1, w)) {
        ok = false;
        break;
      }
      const uint8_t* kb = ring + s * 2 * C::kHalf;
      const uint8_t* vb = kb + C::kHalf;

      // ---- S = Q K^T
      float sc[C::kNT][4];
#pragma unroll
      for (int nt8 = 0; nt8 < C::kNT; ++nt8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt8][e] = 0.f;
        const int row = 8 * nt8 + key_of<C::kPitch>(j);
        if constexpr (C::kCodes) {
#pragma unroll
          for (int ch = 0; ch < D / 64; ++ch) {
            const uint4 u = *reinterpret_cast<const uint4*>(kb + swz<C::kPitch>(row, c + 4 * ch));
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma_16x8x16<true>(sc[nt8], qa[4 * ch + e], c8::decode2_f16(x[e]), c8::decode2_f16(x[e] >> 16));
          }
        } else {
#pragma unroll
          for (int ch = 0; ch < D / 32; ++ch) {
            const uint4 u = *reinterpret_cast<const uint4*>(kb + (ch >> 1) * C::kBlockBytes +
                                                            swz<C::kPitch>(row, c + 4 * (ch & 1)));
            mma_16x8x16<C::kMmaF16>(sc[nt8], qa[2 * ch], u.x, u.y);
            mma_16x8x16<C::kMmaF16>(sc[nt8], qa[2 * ch + 1], u.z, u.w);
          }
        }
      }

      // ---- scale, mask, row maxima
      const int key0 = k0(i);
      const bool edge = key0 + C::kKeys > lim_all;
      float ve[C::kNT][2];  // value exponents of this lane's keys
      float mx_lo = -INFINITY, mx_hi = -INFINITY, mw_lo = -INFINITY, mw_hi = -INFINITY;
#pragma unroll
      for (int nt8 = 0; nt8 < C::kNT; ++nt8)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = 8 * nt8 + key_of<C::kPitch>(2 * c + e);
          float lo = sc[nt8][e] * rs_lo, hi = sc[nt8][2 + e] * rs_hi;
          if constexpr (C::kCodes) {
            const uint32_t x = __shfl_sync(0xffffffffu, exps_now, key & 31) >> (16 * (key >> 5));
            const float kf = c8::scale(x & 0xff);
            ve[nt8][e] = (float)((int)((x >> 8) & 0xff) - 127);
            lo *= kf;
            hi *= kf;
          }
          if (edge) {
            if (key0 + key >= lim_lo) lo = -INFINITY;
            if (key0 + key >= lim_hi) hi = -INFINITY;
          }
          sc[nt8][e] = lo;
          sc[nt8][2 + e] = hi;
          mx_lo = fmaxf(mx_lo, lo);
          mx_hi = fmaxf(mx_hi, hi);
          if constexpr (C::kCodes) {
            mw_lo = fmaxf(mw_lo, lo + ve[nt8][e]);
            mw_hi = fmaxf(mw_hi, hi + ve[nt8][e]);
          }
        }
#pragma unroll
      for (int x = 1; x <= 2; x <<= 1) {
        mx_lo = fmaxf(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, x));
        mx_hi = fmaxf(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, x));
        if constexpr (C::kCodes) {
          mw_lo = fmaxf(mw_lo, __shfl_xor_sync(0xffffffffu, mw_lo, x));
          mw_hi = fmaxf(mw_hi, __shfl_xor_sync(0xffffffffu, mw_hi, x));
        }
      }
      if constexpr (!C::kCodes) {
        mw_lo = mx_lo;
        mw_hi = mx_hi;
      }
      if (__any_sync(0xffffffffu, mx_lo > m_lo || mx_hi > m_hi || mw_lo > mu_lo || mw_hi > mu_hi)) {
        // a maximum grew: rescale (a state at -inf holds zeros; 2^-inf = 0)
        auto grow = [](float& m, float mx) {
          const float m_new = fmaxf(m, mx);
          const float f = m_new == m ? 1.f : ex2_approx(m - m_new);
          m = m_new;
          return f;
        };
        l_lo *= grow(m_lo, mx_lo);
        l_hi *= grow(m_hi, mx_hi);
        const float f_lo = grow(mu_lo, mw_lo), f_hi = grow(mu_hi, mw_hi);
#pragma unroll
        for (int d = 0; d < C::kDT; ++d) {
          acc[d][0] *= f_lo;
          acc[d][1] *= f_lo;
          acc[d][2] *= f_hi;
          acc[d][3] *= f_hi;
        }
      }
      // ---- weights; a row without a key so far (or with -inf scores alone) has reference 0
      const float n_lo = m_lo == -INFINITY ? 0.f : -m_lo, n_hi = m_hi == -INFINITY ? 0.f : -m_hi;
      const float nu_lo = mu_lo == -INFINITY ? 0.f : -mu_lo, nu_hi = mu_hi == -INFINITY ? 0.f : -mu_hi;
      uint32_t pa[C::kNT / 2][4];
#pragma unroll
      for (int nt8 = 0; nt8 < C::kNT; ++nt8) {
        float q_lo[2], q_hi[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p_lo = ex2_approx(sc[nt8][e] + n_lo), p_hi = ex2_approx(sc[nt8][2 + e] + n_hi);
          l_lo += p_lo;  // sums take the unrounded weights
          l_hi += p_hi;
          q_lo[e] = C::kCodes ? ex2_approx(sc[nt8][e] + ve[nt8][e] + nu_lo) : p_lo;
          q_hi[e] = C::kCodes ? ex2_approx(sc[nt8][2 + e] + ve[nt8][e] + nu_hi) : p_hi;
        }
        pa[nt8 / 2][(nt8 & 1) * 2] = pack16x2<C::kMmaF16>(q_lo[0], q_lo[1]);
        pa[nt8 / 2][(nt8 & 1) * 2 + 1] = pack16x2<C::kMmaF16>(q_hi[0], q_hi[1]);
      }

      // ---- u += P V.  At the edge, values of keys past the end become zero, and so
      // do those that are not finite of keys that only some rows see: 0 * NaN would
      // reach the rows that do not.  The rows that do see them get them below.
      bool bad = false;
      auto clean = [&](uint32_t& x, int row) {
        if (key0 + row >= len) {
          x = 0;
        } else if (key0 + row >= lim_all) {
          const uint32_t y = finite_only<Kind>(x);
          bad |= y != x;
          x = y;
        }
      };
#pragma unroll
      for (int kk = 0; kk < C::kNT / 2; ++kk) {
        int row[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) row[r] = 16 * kk + 8 * (r >> 1) + key_of<C::kPitch>(2 * c + (r & 1));
        if constexpr (C::kCodes) {
          constexpr int kWords = C::kRun / 4;
          uint32_t x[4][kWords];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (kWords == 4) {
              const uint4 u = *reinterpret_cast<const uint4*>(vb + swz<C::kPitch>(row[r], block_of(j)));
              x[r][0] = u.x; x[r][1] = u.y; x[r][2] = u.z; x[r][3] = u.w;
            } else {
              const uint2 u = *reinterpret_cast<const uint2*>(vb + swz<C::kPitch>(row[r], j >> 1) + (j & 1) * 8);
              x[r][0] = u.x; x[r][1] = u.y;
            }
            if (edge)
#pragma unroll
              for (int v = 0; v < kWords; ++v) clean(x[r][v], row[r]);
          }
#pragma unroll
          for (int v = 0; v < kWords; ++v) {
            const uint32_t a0 = prmt(x[0][v], x[1][v], 0x5140), a1 = prmt(x[0][v], x[1][v], 0x7362);
            const uint32_t b0 = prmt(x[2][v], x[3][v], 0x5140), b1 = prmt(x[2][v], x[3][v], 0x7362);
            mma_16x8x16<true>(acc[4 * v], pa[kk], c8::decode2_f16(a0), c8::decode2_f16(b0));
            mma_16x8x16<true>(acc[4 * v + 1], pa[kk], c8::decode2_f16(a0 >> 16), c8::decode2_f16(b0 >> 16));
            mma_16x8x16<true>(acc[4 * v + 2], pa[kk], c8::decode2_f16(a1), c8::decode2_f16(b1));
            mma_16x8x16<true>(acc[4 * v + 3], pa[kk], c8::decode2_f16(a1 >> 16), c8::decode2_f16(b1 >> 16));
          }
        } else {
#pragma unroll
          for (int blk = 0; blk < C::kBlocks; ++blk) {
            uint32_t x[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint4 u = *reinterpret_cast<const uint4*>(vb + blk * C::kBlockBytes +
                                                              swz<C::kPitch>(row[r], block_of(j)));
              x[r][0] = u.x; x[r][1] = u.y; x[r][2] = u.z; x[r][3] = u.w;
              if (edge)
#pragma unroll
                for (int v = 0; v < 4; ++v) clean(x[r][v], row[r]);
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              mma_16x8x16<C::kMmaF16>(acc[8 * blk + 2 * v], pa[kk], prmt(x[0][v], x[1][v], 0x5410),
                                      prmt(x[2][v], x[3][v], 0x5410));
              mma_16x8x16<C::kMmaF16>(acc[8 * blk + 2 * v + 1], pa[kk], prmt(x[0][v], x[1][v], 0x7632),
                                      prmt(x[2][v], x[3][v], 0x7632));
            }
          }
        }
      }
      if (edge && __any_sync(0xffffffffu, bad)) {
        // what is not finite goes to the rows that see its key, element by element
        for (int key = max(0, lim_all - key0); key < min(C::kKeys, len - key0); ++key)
#pragma unroll
          for (int run = 0; run < C::kDT / C::kRun; ++run)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int x = 0; x < C::kRun; ++x) {
                const int d = d_of<C>(2 * c + e, run) + x;
                const int byte = d * (C::kCodes ? 1 : 2) % C::kPitch, blk = d * (C::kCodes ? 1 : 2) / C::kPitch;
                const uint8_t* at = vb + blk * C::kBlockBytes + swz<C::kPitch>(key, byte >> 4) + (byte & 15);
                float v;
                if constexpr (C::kCodes)
                  v = c8::decode2(*at).x;
                else if constexpr (C::kMmaF16)
                  v = __half2float(*reinterpret_cast<const __half*>(at));
                else
                  v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at));
                if (!(fabsf(v) < INFINITY)) {
                  if (key0 + key < lim_lo) acc[run * C::kRun + x][e] += v;
                  if (key0 + key < lim_hi) acc[run * C::kRun + x][2 + e] += v;
                }
              }
      }

      // ---- hand the stage back
      __syncwarp();
      if constexpr (WR > 1) {
        if (lane == 0) mbar_arrive(&empty[s]);
      }
      ++taken;
      refill();
      if constexpr (WR > 1) ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    }
    if (!ok && leader) {  // gave up: let the copies in flight land before the memory goes
      for (unsigned g = taken; g < issued; ++g)
        mbar_wait_drain(&full[g % C::kStages], (g / C::kStages) & 1, a.wait_limit_ns);
    }

    // ---- join the key groups and write the run's state
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) {
      l_lo += __shfl_xor_sync(0xffffffffu, l_lo, x);
      l_hi += __shfl_xor_sync(0xffffffffu, l_hi, x);
    }
    const int rl = 16 * wr + j;
    if (c == 0) {
      s_m[wk][rl] = m_lo;
      s_l[wk][rl] = l_lo;
      s_mu[wk][rl] = mu_lo;
      s_m[wk][rl + 8] = m_hi;
      s_l[wk][rl + 8] = l_hi;
      s_mu[wk][rl + 8] = mu_hi;
    }
    __syncthreads();  // every warp is done with its stages: their memory takes the states
    constexpr int kPad = D + 4;
    float* su = reinterpret_cast<float*>(smem);  // [kWK][16 WR][kPad]
#pragma unroll
    for (int run = 0; run < C::kDT / C::kRun; ++run)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* lo = su + (wk * 16 * WR + rl) * kPad + d_of<C>(2 * c + e, run);
#pragma unroll
        for (int x = 0; x < C::kRun; x += 4) {
          float (*v)[4] = acc + run * C::kRun + x;
          if (r_lo < rows) *reinterpret_cast<float4*>(lo + x) = make_float4(v[0][e], v[1][e], v[2][e], v[3][e]);
          if (r_hi < rows)
            *reinterpret_cast<float4*>(lo + 8 * kPad + x) =
                make_float4(v[0][2 + e], v[1][2 + e], v[2][2 + e], v[3][2 + e]);
        }
      }
    __syncthreads();
    const PartSlot slot = own_slot(a, blockIdx.x, tile0 == 0, tile1 == nt, slab, row0, 16 * WR, rows, D);
    const int valid = min(16 * WR, rows - row0);
    for (int idx = threadIdx.x; idx < valid * (D / 4); idx += kOwnThreads) {
      const int r = idx / (D / 4), d = idx % (D / 4) * 4;
      float m = -INFINITY, mu = -INFINITY;
#pragma unroll
      for (int g = 0; g < C::kWK; ++g) {
        m = fmaxf(m, s_m[g][r]);
        mu = fmaxf(mu, s_mu[g][r]);
      }
      float l = 0.f;
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < C::kWK; ++g) {
        l += s_l[g][r] * join_factor(s_m[g][r], m);
        const float f = join_factor(s_mu[g][r], mu);
        const float4 v = *reinterpret_cast<const float4*>(su + (g * 16 * WR + r) * kPad + d);
        u.x += v.x * f;
        u.y += v.y * f;
        u.z += v.z * f;
        u.w += v.w * f;
      }
      *reinterpret_cast<float4*>(slot.u + (long long)r * D + d) = u;
      if (d == 0) slot.ml[r] = make_float4(m, l, mu, 0.f);
    }
    fence_proxy_async_smem();  // the next run's copies write where the states were read
    __syncthreads();
    t += tile1 - tile0;
  }
  // this kernel's end has to mean the end of the pass over the prefix too
  if (threadIdx.x == 0) grid_wait();
}

template <int Kind, int D, int WR>
cudaError_t launch_own_w(const ServeArgs& a, bool q_f16, bool after, cudaStream_t s) {
  using C = OwnCfg<Kind, D, WR>;
  OwnParams p;
  p.a = a;
  p.q_f16 = q_f16;
  p.row_groups = (a.group * a.nq + 16 * WR - 1) / (16 * WR);
  const uint64_t slabs = (uint64_t)a.B * a.Hk;
  if (!make_map_cache(&p.tk, a.k, C::kCodes ? 1 : 2, D, a.cap, slabs, C::kKeys) ||
      !make_map_cache(&p.tv, a.v, C::kCodes ? 1 : 2, D, a.cap, slabs, C::kKeys))
    return note_error("cache tensor map encode", cudaErrorInvalidValue);
  const cudaError_t e = cudaFuncSetAttribute(own_kernel<Kind, D, WR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return note_error("cached decoding smem attribute", e);
  return note_error("cached decoding launch",
                    launch_serve_kernel(own_kernel<Kind, D, WR>, kOwnCtas, kOwnThreads, C::kSmem, after, s, p));
}

template <int Kind>
cudaError_t launch_own_k(const ServeArgs& a, int D, bool q_f16, bool after, cudaStream_t s) {
  // Row tiles of 16: a CTA holds 1, 2 or 4.  More row tiles mean fewer key groups to
  // share the stream, so a CTA takes as many as the rows fill.
  const int wr = own_row_tiles(a.group * a.nq);
  if (D == 64) {
    if (wr == 1) return launch_own_w<Kind, 64, 1>(a, q_f16, after, s);
    if (wr == 2) return launch_own_w<Kind, 64, 2>(a, q_f16, after, s);
    return launch_own_w<Kind, 64, 4>(a, q_f16, after, s);
  }
  if (wr == 1) return launch_own_w<Kind, 128, 1>(a, q_f16, after, s);
  if (wr == 2) return launch_own_w<Kind, 128, 2>(a, q_f16, after, s);
  return launch_own_w<Kind, 128, 4>(a, q_f16, after, s);
}

}  // namespace
}  // namespace fa
