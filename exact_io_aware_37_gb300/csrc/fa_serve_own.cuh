// The pass over the sequences' own cache rows of a decoding step
// (fa_decode_cache, fa_decode_shared).
//
// Mathematics.  For the query rows of one (sequence, key head) -- group * nq of
// them, at most R a CTA -- and tiles of 128 keys: S^T = K Q^T, P^T = 2^(c2 S - ref),
// O^T += V^T P^T, with a running reference for the maximum.  The tile of keys is
// the 128-row operand of both products, the query rows are the narrow one, so
// one or sixty query rows cost a tensor core the same and nothing is padding
// but the narrow side's last columns.
//
// The 8-bit cache goes into the products as it is (e4m3, kind::f8f6f4).  A query
// row is scaled by a power of two and held as three e4m3 terms, x = c0 + c1 / 32 +
// c2 / 1024 (12 bits, more than fp16 or bf16 have), each a column of the narrow operand; so
// are the weights, rounded to fp16 first.  A key's power of two multiplies its scores, a value's power of
// two, 2^e, its weight: the weight that is rounded is 2^(s + e - ref_w), with a reference for
// s + e of its own, so that the largest contribution, not the largest weight, sits
// at the top of the terms' range however unlike the rows' scales are.  The
// normaliser sums the unrounded 2^(s - ref_l).
//
// Bound.  Every cache row is read once: HBM.  Per 128 keys of D = 128 codes the
// tensor core spends 256 cycles, the copies at the full rate 1400: B16 H32 8192 keys D128 take 160 us a step (6.7
// TB/s).  24 sequences of up to 16384 keys, 8 key heads, 60 us at the copy rate, take 71 at 4 query rows a key head,
// 72 at 8, 76 at 16, 84 at 20, 85 at 24: there the softmax warps issue 38 % of the SM's slots and wait for the rest.  (The products
// by warp-level MMA were tried first: about 60 cycles each a warp on this part, so eight
// warps an SM held the step at 239 us, B16 H32 8192 keys D128.)
//
// Roles (6 warps).  Warps 0-3: softmax, one key (its S^T lane) a thread.  A tile is
// weighed with the references as they are; only if some score outgrew them, which one
// barrier with a vote finds out, are new ones found and the tile weighed again.  The threads
// write P^T as the second product's narrow operand, in one of two places, so that the next
// tile is weighed while that product runs, and read O^T at a run's end, by when the next
// run's queries are in place.  Warp 4: TMA producer; K and V tiles share one ring that runs
// on over a CTA's runs.  Warp 5: MMA issuer; S^T of the next tile is issued before the
// softmax of this one is done.
//
// Schedule.  The tiles of all (sequence, head, row group) units are laid out in
// a row and cut into equal shares, one a CTA, from the lengths on the device; a run is
// what a share holds of one unit.  A unit that is cut leaves one state a run, joined by the merge kernel.
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

constexpr int kOwnThreads = 192;
constexpr int kOwnTmaWarp = 4, kOwnMmaWarp = 5;
constexpr int kBoxKeys = 32;  // keys of one TMA box: a last tile reads no more boxes than it has keys for
// Weights enter the terms times 2^4 and may outgrow their reference by 2^4, so that
// they stay within 256 and the terms reach down to 2^-20 / 2^4 = 2^-24 of the reference (fp16:
// 2^-25).  A slack of 2^1 at a scale of 2^7 found new references in every other tile
// at 20 rows a key head and nearly doubled the step.
constexpr float kWeightLog2 = 4.f;  // codes only
constexpr float kRefSlack = 4.f;   // log2 units a weight may outgrow its reference by
constexpr float kSumSlack = 60.f;  // the same for the float32 normaliser

struct OwnParams {
  CUtensorMap tk, tv;
  ServeArgs a;
  int row_groups;
  bool q_f16;  // 8-bit cache: the queries' type (16-bit caches have the queries' type)
};

enum CacheKind { kE4m3, kBf16, kF16 };

template <int Kind, int D, int R>
struct OwnCfg {
  static constexpr bool kCodes = Kind == kE4m3;
  static constexpr int kElem = kCodes ? 1 : 2;
  static constexpr int kRowBytes = D * kElem;
  static constexpr int kPitch = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row in one swizzled block
  static constexpr int kBlocks = kRowBytes / kPitch;                // blocks side by side (D = 128 in 16 bits: 2)
  static constexpr int kBlockBytes = kOwnTile * kPitch;
  static constexpr int kTileBytes = kOwnTile * kRowBytes;
  static constexpr int kTerms = kCodes ? 3 : 1;
  static constexpr int kN = (R * kTerms + 15) / 16 * 16;  // columns of the narrow operand; term x of row r is x R + r
  static constexpr int kQBlock = kN * kPitch;             // Q: the same blocks, kN rows
  // P^T.  Codes: a key's weights together, 32 columns of all keys a block (MN-major, 32-byte swizzle), so that a
  // thread stores eight rows' bytes of a term at once (a byte a row and term, K-major: 94 us a step, so
  // 88, 24 sequences of up to 16384 keys, 20 query rows a key head).  16-bit: a row's 128 weights together, in two blocks.
  static constexpr int kPN = kCodes ? (kN + 31) / 32 * 32 : kN;  // columns of the second product
  static constexpr int kPBlock = kCodes ? kOwnTile * 32 : kN * 128;
  static constexpr int kPBytes = ((kCodes ? kPN / 32 : 2) * kPBlock + 1023) / 1024 * 1024;
  static constexpr int kPOff = 0;  // two: the next tile is weighed while a product reads this one's
  static constexpr int kQOff = 2 * kPBytes;
  static constexpr int kRingOff = kQOff + (kBlocks * kQBlock + 1023) / 1024 * 1024;
  // at D = 64 the second half of V^T's 128 rows is read from what follows V (its products go to
  // tensor-memory lanes that nothing reads); past the ring's last slot that is this many bytes
  static constexpr int kPad = D == 64 ? kTileBytes : 0;
  // as many slots as leave room for a second CTA on the SM (228 KB; each also takes 1 KB of the
  // system's, 1 KB for alignment and up to 3 KB below), if that is three (a third CTA, at the same
  // bytes in flight, gained nothing).  No more than 80 KB: of four, five and six slots of 16 KB five are the fastest or
  // within 0.3 us of it over 15 shapes (B16 H32 8192 keys: four 1.5 % slower, six 1.3 %; B24 of up to 16384 keys, 8 key heads, 8 rows: 1.5 and 3 %).
  static constexpr int kFit = (108 * 1024 - kRingOff - kPad) / kTileBytes;
  static constexpr int kPerSm = kFit >= 3 ? 2 : 1;
  static constexpr int kMost = kTileBytes <= 8192 ? 8 : 5;
  // K of step g: slot 2 g, V: 2 g + 1, modulo kSlots
  static constexpr int kSlots = kFit >= 3 ? (kFit < kMost ? kFit : kMost) : 6;
  static constexpr int kSmem = kRingOff + kSlots * kTileBytes + kPad + 1024;
  static constexpr int kCols = 2 * kN + kPN <= 64 ? 64 : 2 * kN + kPN <= 128 ? 128 : 256;  // two S^T, O^T
  static constexpr int kChunk = R < 8 ? R : 8;                                 // rows read out together
};

// Byte offset of 16-byte chunk `chunk` of row `row` in a swizzled block.
template <int kPitch>
__device__ __forceinline__ int swz(int row, int chunk) {
  if constexpr (kPitch == 128)
    return row * 128 + ((chunk ^ (row & 7)) << 4);
  else
    return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

template <int Kind>
__device__ __forceinline__ float cache_value(const uint8_t* p) {
  if constexpr (Kind == kE4m3) return c8::decode2(*p).x;
  if constexpr (Kind == kBf16) return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
  if constexpr (Kind == kF16) return __half2float(*reinterpret_cast<const __half*>(p));
}

// Elements of a word of values that are not finite become zero.
template <int Kind>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if constexpr (Kind != kE4m3) return finite_only16<Kind == kF16>(w);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (((w >> (8 * i)) & 0x7fu) == 0x7fu) w &= ~(0xffu << (8 * i));
  return w;
}

// Sums of R values a lane over the warp: l[0] of lane x becomes the sum of value x % R2,
// R2 the power of two from R on (values past R count as 0).  R2 - 1 + log2(32 / R2) shuffles, not 5 R.
template <int R>
__device__ __forceinline__ void sum_rows(float (&l)[R], int lane) {
  constexpr int R2 = R <= 4 ? 4 : R <= 8 ? 8 : R <= 16 ? 16 : 32;
#pragma unroll
  for (int half = R2 / 2; half >= 1; half >>= 1) {
    const bool up = (lane & half) != 0;
#pragma unroll
    for (int r = 0; r < half; ++r) {
      const float a = r < R ? l[r] : 0.f, b = r + half < R ? l[r + half] : 0.f;
      const float got = __shfl_xor_sync(0xffffffffu, up ? a : b, half);
      if (r < R) l[r] = (up ? b : a) + got;
    }
  }
#pragma unroll
  for (int m = R2; m < 32; m <<= 1) l[0] += __shfl_xor_sync(0xffffffffu, l[0], m);
}

// What the threads share about two query rows of a run (x and y; two, for the packed float32 arithmetic).
struct RowPair {
  float2 factor;  // from products to log2 units
  float2 neg_w;   // minus the references (neg_w holds the weights' scale)
  float2 neg_l;
  int2 limit;     // keys they see
};
// In place of minus a reference while a row has seen no score above -inf: any such score
// outgrows it.
constexpr float kNoReference = 1e30f;

template <int Kind, int D, int R>
__global__ void __launch_bounds__(kOwnThreads, OwnCfg<Kind, D, R>::kPerSm) own_kernel(
    const __grid_constant__ OwnParams p) {
  using C = OwnCfg<Kind, D, R>;
  constexpr unsigned H = C::kSlots;
  constexpr float kWeightScale = C::kCodes ? kWeightLog2 : 0.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // Steps (tiles) g are counted over all of a CTA's runs.  full / free: the ring; bar_s[g % 2]:
  // S^T(g) complete; bar_p[g % 2]: P^T(g) written and S^T(g) read out (the MMA thread has waited
  // for it before it issues S^T(g + 2) over the same columns); bar_o[g % 2]: O^T += (g) complete (S^T(g)
  // is issued behind O^T += (g - 2), so with bar_s P^T(g)'s place is free, and bar_o's phase before this
  // one over); bar_q: a run's Q written.
  __shared__ __align__(8) uint64_t bar_full[H], bar_free[H];
  __shared__ __align__(8) uint64_t bar_s[2], bar_p[2], bar_o[2], bar_q, bar_done;
  // by the run's parity: the next run's are written while this one's are in use
  __shared__ __align__(16) RowPair s_row[2][R / 2];
  __shared__ float s_refw[2][R], s_refl[2][R];  // references of the weights and of the normaliser
  __shared__ float s_mw[4][R], s_ml[4][R];      // warps' maxima
  __shared__ float s_sum[4][R];                 // and sums, at a run's end
  __shared__ float s_fw[R], s_fl[R];            // rescaling
  __shared__ int s_bad[2];
  __shared__ OwnPlan plan;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;

  const ServeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = a.group * a.nq;

  if (threadIdx.x == 0) {
    for (unsigned s = 0; s < H; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_free[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar_s[s], 1);
      mbar_init(&bar_p[s], 4);
      mbar_init(&bar_o[s], 1);
    }
    mbar_init(&bar_q, 4);
    mbar_init(&bar_done, 1);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
  }
  if (warp == kOwnMmaWarp) {
    tmem_alloc(&tmem_base_sh, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  own_plan<kOwnThreads>(a, p.row_groups, plan);  // holds block-wide barriers
  tc_fence_after();
  grid_launch_dependents();
  const uint32_t tmem = tmem_base_sh;
  const WaitCtx w{&abort_flag, a.status, a.wait_limit_ns};

  // ---- the CTA's runs, walked alike by every role
  struct Run {
    int len, row0, slab, tile0, n;
    bool ends;  // the run holds the unit's last tile
  };
  struct Walk {  // the next unit, and where in its cost the share goes on (0 but for the first)
    long long t;
    int b, hk, rg, off;
  };
  auto next_run = [&](Walk& k, Run& q) -> bool {
    while (k.t < plan.end) {
      q.len = seq_len(a, k.b);
      const int nt = own_tiles(q.len), cost = own_cost(a, nt);
      if (cost == 0) {  // an empty sequence
        ++k.b;
        continue;
      }
      const int x0 = k.off, x1 = (int)min((long long)cost, x0 + (plan.end - k.t));
      k.t += x1 - x0;
      q.tile0 = max(0, x0 - a.run_cost);
      q.n = max(0, x1 - a.run_cost) - q.tile0;
      q.ends = x1 == cost;
      q.row0 = k.rg * R;
      q.slab = k.b * a.Hk + k.hk;
      k.off = 0;
      if (++k.rg == p.row_groups) {
        k.rg = 0;
        if (++k.hk == a.Hk) {
          k.hk = 0;
          ++k.b;
        }
      }
      if (q.n > 0) return true;  // else the share ended before the unit's first tile
    }
    return false;
  };
  Walk walk{plan.first, plan.b, plan.hk, plan.rg, plan.off};

  if (warp < 4) {
    // ------------------------------------------------------------ softmax
    const int tid = threadIdx.x;  // the key of a tile that this thread holds
    const uint32_t t_s = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t t_o = t_s + 2 * C::kN;
    uint8_t* sq = smem + C::kQOff;
    constexpr int kRowThreads = D / 8;  // threads of a query row, 8 elements each
    constexpr int kPass = 128 / kRowThreads, kPasses = (R + kPass - 1) / kPass;
    const int qr = tid / kRowThreads, qx = tid % kRowThreads * 8;

    auto row_of = [&](auto field, int par, int r) -> auto& {
      auto& two = s_row[par][r >> 1].*field;
      return r & 1 ? two.y : two.x;
    };
    // ---- a run's queries: loaded early, put in place later
    uint4 qv[kPasses];
    auto load_q = [&](const Run& q) {
      const int valid = min(R, rows - q.row0);
#pragma unroll
      for (int x = 0; x < kPasses; ++x) {
        const int r = x * kPass + qr;
        qv[x] = r < valid ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                            ((long long)q.slab * rows + q.row0 + r) * D + qx)
                          : make_uint4(0, 0, 0, 0);
      }
    };
    // The narrow operand of S^T and what the rows' threads share; every S^T of the run before is complete.
    auto put_q = [&](const Run& q, int par) {
      const int valid = min(R, rows - q.row0);
#pragma unroll
      for (int x = 0; x < kPasses; ++x) {
        const int r = x * kPass + qr;
        float factor = a.c2;
        if constexpr (C::kCodes) {
          const uint32_t v[4] = {qv[x].x, qv[x].y, qv[x].z, qv[x].w};
          float f[8], big = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = p.q_f16 ? __half22float2(*reinterpret_cast<const __half2*>(&v[e]))
                                     : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v[e]));
            f[2 * e] = y.x;
            f[2 * e + 1] = y.y;
            big = fmaxf(big, fmaxf(c8::finite_abs(y.x), c8::finite_abs(y.y)));
          }
#pragma unroll
          for (int m = kRowThreads / 2; m >= 1; m >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
          // Scaled by a power of two to between 112 and 224 (infinities become NaN).  The terms' last step is 2^-19,
          // so an element is off by at most 2^-20 there (and 2^-25 in fp16), 2^-26 of the row's largest: float32's own
          // products lose as much where the largest counts, and where it meets zeros a row needs channels
          // 2^16 apart before it shows beside a score's other roundings.
          const int eb = c8::exp_byte(big);
          const float scale = 0.5f * c8::inv_scale(eb);
          factor *= 2.f * c8::scale(eb);
          uint32_t t[4][3];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float lo = f[2 * e] * scale, hi = f[2 * e + 1] * scale;
            lo = fabsf(lo) < INFINITY ? lo : __uint_as_float(0x7fffffffu);
            hi = fabsf(hi) < INFINITY ? hi : __uint_as_float(0x7fffffffu);
            c8::encode2_terms(__floats2half2_rn(lo, hi), t[e]);
          }
          if (r < R)
#pragma unroll
            for (int k = 0; k < 3; ++k)
              *reinterpret_cast<uint2*>(sq + swz<C::kPitch>(k * R + r, qx >> 4) + (qx & 15)) =
                  make_uint2(t[0][k] | t[1][k] << 16, t[2][k] | t[3][k] << 16);
        } else if (r < R) {
          *reinterpret_cast<uint4*>(sq + (qx >> 6) * C::kQBlock + swz<C::kPitch>(r, (qx & 63) >> 3)) = qv[x];
        }
        if (r < R && qx == 0) {
          // a row past the last weighs nothing and outgrows nothing
          const bool there = r < valid;
          const int limit = a.causal ? max(0, q.len - a.nq + (q.row0 + r) % a.nq + 1) : q.len;
          row_of(&RowPair::factor, par, r) = factor;
          row_of(&RowPair::neg_w, par, r) = row_of(&RowPair::neg_l, par, r) = there ? kNoReference : -INFINITY;
          row_of(&RowPair::limit, par, r) = limit;
          s_refw[par][r] = s_refl[par][r] = there ? -INFINITY : INFINITY;
        }
      }
      if (tid == 0) s_bad[par] = 0;
      fence_proxy_async_smem();
      named_bar_sync(1, 128);
      if (lane == 0) mbar_arrive(&bar_q);
    };

    int ek = 0, ev = 0;  // exponents of this thread's key, loaded a tile ahead
    auto load_exps = [&](const Run& q, int i) {
      const int key = (q.tile0 + i) * kOwnTile + tid;
      if (C::kCodes && key < q.len) {
        const long long at = (long long)q.slab * a.cap + key;
        ek = __ldg(a.k_exp + at);
        ev = __ldg(a.v_exp + at);
      }
    };
    // Scores of a chunk of rows as they leave the products (codes: the three terms joined).
    auto read_chunk = [&](uint32_t at, float (&v)[C::kChunk]) {
      uint32_t x[C::kTerms][C::kChunk];
#pragma unroll
      for (int k = 0; k < C::kTerms; ++k) tmem_ld(at + k * R, x[k]);
#pragma unroll
      for (int k = 0; k < C::kTerms; ++k) tmem_ld_wait(x[k]);
#pragma unroll
      for (int e = 0; e < C::kChunk; e += 2) {
        auto as = [&](int k, int i) { return __uint_as_float(x[k][e + i]); };
        v[e] = as(0, 0);
        v[e + 1] = as(0, 1);
        if constexpr (C::kCodes) {
          float lo, hi;
          ffma2(lo, hi, as(2, 0), as(2, 1), c8::kTerm, as(1, 0), as(1, 1));
          ffma2(v[e], v[e + 1], lo, hi, c8::kTerm, v[e], v[e + 1]);
        }
      }
    };

    bool ok = true;
    unsigned g = 0;
    int par = 0;
    Run q, nx;
    bool have = next_run(walk, q);
    if (have) {
      load_q(q);
      load_exps(q, 0);
      put_q(q, 0);
    }
    while (ok && have) {
      const int valid = min(R, rows - q.row0);
      const int lim_all = a.causal ? max(0, q.len - a.nq + 1) : q.len;  // keys that every row sees
      const RowPair* row = s_row[par];
      float l[R];  // this thread's share of the normaliser
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = 0.f;

      for (int i = 0; i < q.n; ++i, ++g) {
        const int key0 = (q.tile0 + i) * kOwnTile, key = key0 + tid;
        const float kf = C::kCodes ? c8::scale(ek) : 1.f;
        const float ve = C::kCodes ? (float)(ev - 127) : 0.f;
        if (i + 1 < q.n) {
          load_exps(q, i + 1);
        } else {
          have = next_run(walk, nx);
          if (have) {
            load_q(nx);
            load_exps(nx, 0);
          }
        }
        // A wait that gives up leaves its warp in step until the next vote, where all
        // four warps stop together: none may be left alone at a barrier.
        ok = ok && warp_wait(&bar_s[g & 1], (g >> 1) & 1, w);
        tc_fence_after();
        const uint32_t at_s = t_s + (g & 1) * C::kN;
        uint8_t* sp = smem + C::kPOff + (g & 1) * C::kPBytes;
        const bool edge = key0 + kOwnTile > lim_all;
        // At the edge: values of keys past the end become zero, and so do those that are
        // not finite of keys that only some rows see (0 * NaN would reach the rows that
        // do not); the rows that do see them get them at the run's end.
        if (edge && key >= lim_all) {
          const unsigned h = 2 * g + 1;
          uint8_t* v = smem + C::kRingOff + (h % H) * C::kTileBytes;
          if (!mbar_wait(&bar_full[h % H], (h / H) & 1, w))
            ok = false;
          else
            for (int blk = 0; blk < C::kBlocks; ++blk)
              for (int ch = 0; ch < C::kPitch / 16; ++ch) {
                uint4* at = reinterpret_cast<uint4*>(v + blk * C::kBlockBytes + swz<C::kPitch>(tid, ch));
                if (key >= q.len) {
                  *at = make_uint4(0, 0, 0, 0);
                } else {
                  const uint4 u = *at;
                  const uint4 y = make_uint4(finite_only<Kind>(u.x), finite_only<Kind>(u.y), finite_only<Kind>(u.z),
                                             finite_only<Kind>(u.w));
                  if (u.x != y.x || u.y != y.y || u.z != y.z || u.w != y.w) {
                    *at = y;
                    s_bad[par] = 1;
                  }
                }
              }
        }
        // Finds the rows' references again: false when some warp has given up.
        auto refer = [&]() -> bool {
#pragma unroll 1
          for (int r0 = 0; r0 < valid; r0 += C::kChunk) {
            float v[C::kChunk];
            read_chunk(at_s + r0, v);
#pragma unroll
            for (int e = 0; e < C::kChunk; ++e) {
              float x = v[e] * (row_of(&RowPair::factor, par, r0 + e) * kf);
              if (edge && key >= row_of(&RowPair::limit, par, r0 + e)) x = -INFINITY;
              const float mw = warp_max(x + ve), ml = C::kCodes ? warp_max(x) : mw;
              if (lane == 0) {
                s_mw[warp][r0 + e] = mw;
                s_ml[warp][r0 + e] = ml;
              }
            }
          }
          if (!named_bar_and(1, 128, ok)) return false;
          if (tid < valid) {
            auto grow = [](float& ref, float m0, float m1, float m2, float m3) {
              const float m = fmaxf(ref, fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)));
              const float f = m == ref ? 1.f : exp2f(ref - m);
              ref = m;
              return f;
            };
            s_fw[tid] = grow(s_refw[par][tid], s_mw[0][tid], s_mw[1][tid], s_mw[2][tid], s_mw[3][tid]);
            s_fl[tid] = grow(s_refl[par][tid], s_ml[0][tid], s_ml[1][tid], s_ml[2][tid], s_ml[3][tid]);
            const float rw = s_refw[par][tid], rl = s_refl[par][tid];
            row_of(&RowPair::neg_w, par, tid) = rw == -INFINITY ? kNoReference : kWeightScale - rw;
            row_of(&RowPair::neg_l, par, tid) = rl == -INFINITY ? kNoReference : -rl;
          }
          named_bar_sync(1, 128);
          return true;
        };
        // Weighs the tile.  kFirst: adds to the sums (unrounded weights) and says whether some
        // score outgrew its reference.  Again, under new references: the sums, rescaled, hold
        // the tile already, but where the old reference let a weight overflow; what was there before
        // is then nothing beside it.
        auto weigh = [&](auto at_edge, auto first) -> bool {
          float most_w = -INFINITY, most_l = -INFINITY;
#pragma unroll
          for (int r0 = 0; r0 < R; r0 += C::kChunk) {
            if (r0 >= valid) break;
            float v[C::kChunk];
            uint32_t t[C::kChunk / 2][C::kTerms];
            read_chunk(at_s + r0, v);
#pragma unroll
            for (int e = 0; e < C::kChunk; e += 2) {
              const RowPair two = row[(r0 + e) / 2];
              const bool hide0 = at_edge.value && key >= two.limit.x, hide1 = at_edge.value && key >= two.limit.y;
              float2 f = two.factor, nw = two.neg_w;
              if constexpr (C::kCodes) {
                fmul2(f.x, f.y, f.x, f.y, kf, kf);
                fadd2(nw.x, nw.y, ve, ve);
              }
              float x0, x1, sum0, sum1;
              ffma2(x0, x1, v[e], v[e + 1], f, nw);
              if (hide0) x0 = -INFINITY;
              if (hide1) x1 = -INFINITY;
              if constexpr (C::kCodes) {
                float y0, y1;
                ffma2(y0, y1, v[e], v[e + 1], f, two.neg_l);
                if (hide0) y0 = -INFINITY;
                if (hide1) y1 = -INFINITY;
                sum0 = ex2_approx(y0);
                sum1 = ex2_approx(y1);
                if (first.value) most_l = fmaxf(most_l, fmaxf(y0, y1));
              }
              if (first.value) most_w = fmaxf(most_w, fmaxf(x0, x1));
              v[e] = ex2_approx(x0);
              v[e + 1] = ex2_approx(x1);
              if constexpr (!C::kCodes) {
                sum0 = v[e];
                sum1 = v[e + 1];
              }
              if (first.value) {
                fadd2(l[r0 + e], l[r0 + e + 1], sum0, sum1);
              } else {
                if (l[r0 + e] == INFINITY) l[r0 + e] = sum0;
                if (l[r0 + e + 1] == INFINITY) l[r0 + e + 1] = sum1;
              }
            }
#pragma unroll
            for (int e = 0; e < C::kChunk; e += 2) {
              if constexpr (C::kCodes)
                c8::encode2_terms(__floats2half2_rn(v[e], v[e + 1]), t[e / 2]);
              else  // the queries' type, as the operands of one product have one type; the normaliser is not rounded
                t[e / 2][0] = pack16x2<Kind == kF16>(v[e], v[e + 1]);
            }
            if constexpr (C::kCodes) {
#pragma unroll
              for (int k = 0; k < 3; ++k) {
                const int col = k * R + r0;
                uint8_t* dst = sp + col / 32 * C::kPBlock + tid * 32 + ((col >> 4 ^ tid >> 2) & 1) * 16 + (col & 15);
                if constexpr (C::kChunk == 8)
                  *reinterpret_cast<uint2*>(dst) =
                      make_uint2(__byte_perm(t[0][k], t[1][k], 0x5410), __byte_perm(t[2][k], t[3][k], 0x5410));
                else
                  *reinterpret_cast<uint32_t*>(dst) = __byte_perm(t[0][k], t[1][k], 0x5410);
              }
            } else {
#pragma unroll
              for (int e = 0; e < C::kChunk; e += 2) {
                const int r = r0 + e;
                if (r >= valid) break;
                uint8_t* dst = sp + (tid >> 6) * C::kPBlock + (tid & 7) * 2;
                *reinterpret_cast<uint16_t*>(dst + swz<128>(r, (tid & 63) >> 3)) = (uint16_t)t[e / 2][0];
                *reinterpret_cast<uint16_t*>(dst + swz<128>(r + 1, (tid & 63) >> 3)) = (uint16_t)(t[e / 2][0] >> 16);
              }
            }
          }
          return most_w > kWeightScale + kRefSlack || most_l > kSumSlack;
        };
        auto weigh_tile = [&](auto first) {  // (a second weighing is rare: one form of it will do)
          return edge || !first.value ? weigh(Flag<true>{}, first) : weigh(Flag<false>{}, first);
        };

        ok = __all_sync(0xffffffffu, ok) != 0;
        if (i == 0) {
          if (!refer()) {
            ok = false;
            break;
          }
          weigh_tile(Flag<true>{});
        } else {
          const bool over = weigh_tile(Flag<true>{});
          if (named_bar_or(1, 128, over || !ok)) {
            // O^T is at rest once the last step has been added
            ok = ok && warp_wait(&bar_o[(g - 1) & 1], ((g - 1) >> 1) & 1, w);
            tc_fence_after();
            if (!refer()) {
              ok = false;
              break;
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (r < valid && l[r] != INFINITY) l[r] *= s_fl[r];
#pragma unroll 1
            for (int k = 0; k < C::kTerms; ++k)
#pragma unroll 1
              for (int r0 = 0; r0 < valid; r0 += C::kChunk) {
                uint32_t o[C::kChunk];
                tmem_ld(t_o + k * R + r0, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < C::kChunk; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * s_fw[r0 + e]);
                tmem_st(t_o + k * R + r0, o);
              }
            tmem_st_wait();
            weigh_tile(Flag<false>{});
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[g & 1]);
      }
      // ---- the next run's queries, while this one's last product runs
      const unsigned last = g - 1;
      if (!named_bar_and(1, 128, ok)) break;
      if (have) put_q(nx, par ^ 1);
      ok = named_bar_and(1, 128, warp_wait(&bar_o[last & 1], (last >> 1) & 1, w));
      if (!ok) break;
      tc_fence_after();

      // ---- the run's state
      const long long row_at = (long long)q.slab * rows + q.row0;
      const PartSlot slot = own_slot(a, blockIdx.x, q.tile0 == 0, q.ends, row_at, R, D);
      if (tid < D) {  // whole warps: lane = element of the head width
        const bool bad = s_bad[par] != 0;
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += C::kChunk) {
          if (r0 >= valid) break;
          float v[C::kChunk];
          read_chunk(t_o + r0, v);
#pragma unroll
          for (int e = 0; e < C::kChunk; ++e) {
            const int r = r0 + e;
            if (r >= valid) break;
            float u = C::kCodes ? v[e] * (1.f / (1 << (int)kWeightLog2)) : v[e];
            if (bad) {  // what is not finite of keys that not all rows see
              const int k0 = max(lim_all, q.tile0 * kOwnTile);
              const int k1 = min(row_of(&RowPair::limit, par, r), (q.tile0 + q.n) * kOwnTile);
              for (int key = k0; key < k1; ++key) {
                const float y = cache_value<Kind>(static_cast<const uint8_t*>(a.v) +
                                                  (((long long)q.slab * a.cap + key) * D + tid) * C::kElem);
                if (!(fabsf(y) < INFINITY)) u += y;
              }
            }
            slot.u[(long long)r * D + tid] = u;
          }
        }
      }
      // The rows' sums over the keys: at every step a lane passes half of its rows on and keeps
      // the other half's sums, so that in the end lane x has row x of the first kRows2 rows
      // (lanes that share a row hold equal sums).
      sum_rows<R>(l, lane);
      constexpr int kRows2 = R <= 4 ? 4 : R <= 8 ? 8 : R <= 16 ? 16 : 32;
      if (lane < R && lane < kRows2) s_sum[warp][lane] = l[0];
      named_bar_sync(1, 128);
      if (tid < valid)
        slot.ml[tid] = make_float4(s_refl[par][tid], s_sum[0][tid] + s_sum[1][tid] + s_sum[2][tid] + s_sum[3][tid],
                                   s_refw[par][tid], 0.f);
      tc_fence_before();
      q = nx;
      par ^= 1;
    }
  } else if (warp == kOwnTmaWarp && lane == 0) {
    // ------------------------------------------------------------ producer
    unsigned h = 0;  // tiles of K and V asked for
    bool ok = true;
    Run q;
    while (ok && next_run(walk, q)) {
      for (int i = 0; ok && i < q.n; ++i) {
        const int key0 = (q.tile0 + i) * kOwnTile;
        const int boxes = min(kOwnTile / kBoxKeys, (q.len - key0 + kBoxKeys - 1) / kBoxKeys);
        for (int x = 0; x < 2; ++x, ++h) {
          const unsigned s = h % H;
          if (h >= H && !mbar_wait(&bar_free[s], (h / H - 1) & 1, w)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bar_full[s], boxes * kBoxKeys * C::kRowBytes);
          uint8_t* dst = smem + C::kRingOff + s * C::kTileBytes;
          for (int blk = 0; blk < C::kBlocks; ++blk)
            for (int y = 0; y < boxes; ++y)
              tma_load_3d(dst + blk * C::kBlockBytes + y * kBoxKeys * C::kPitch, x ? &p.tv : &p.tk, &bar_full[s],
                          blk * 64, key0 + y * kBoxKeys, q.slab);
        }
      }
    }
    if (abort_flag)  // let copies already in flight land before the CTA's memory is released
      for (unsigned x = h > H ? h - H : 0; x < h; ++x)
        mbar_wait_drain(&bar_full[x % H], (x / H) & 1, a.wait_limit_ns);
  } else if (warp == kOwnMmaWarp && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    constexpr int kStep = C::kCodes ? 32 : 16;  // elements of one MMA's reduction
    constexpr uint32_t id_s = C::kCodes ? idesc_e4m3(128, C::kN, false, false) : idesc16<Kind == kF16>(128, C::kN, false, false);
    constexpr uint32_t id_o = C::kCodes ? idesc_e4m3(128, C::kPN, true, true) : idesc16<Kind == kF16>(128, C::kN, true, false);
    auto desc = [](const uint8_t* at, uint32_t lbo) {
      return C::kPitch == 128 ? sdesc_sw128(smem_u32(at), lbo, 1024) : sdesc_sw64(smem_u32(at), lbo, 512);
    };
    auto mma = [](uint32_t d, uint64_t x, uint64_t y, uint32_t id, bool acc) {
      if constexpr (C::kCodes)
        mma_f8_ss(d, x, y, id, acc ? 1u : 0u);
      else
        mma_ss(d, x, y, id, acc ? 1u : 0u);
    };
    const uint64_t dk0 = desc(smem + C::kRingOff, 16);
    const uint64_t dv0 = desc(smem + C::kRingOff, C::kBlockBytes);  // V^T: MN-major, the next elements a block further
    const uint64_t dq0 = desc(smem + C::kQOff, 16);
    const uint64_t dp0 = C::kCodes ? sdesc_sw32(smem_u32(smem + C::kPOff), C::kPBlock, 256)
                                   : sdesc_sw128(smem_u32(smem + C::kPOff), 16, 1024);  // of even steps
    bool ok = true;
    unsigned g = 0;
    int run = 0;
    Run q, nx;
    // O^T += V^T P^T of step x
    auto add = [&](unsigned x, bool acc) -> bool {
      const unsigned h = 2 * x + 1, s = h % H;
      if (!mbar_wait(&bar_full[s], (h / H) & 1, w) || !mbar_wait(&bar_p[x & 1], (x >> 1) & 1, w)) return false;
      tc_fence_after();
      const uint64_t v = dv0 + ((s * C::kTileBytes) >> 4), pt = dp0 + (((x & 1) * C::kPBytes) >> 4);
#pragma unroll
      for (int k = 0; k < kOwnTile / kStep; ++k) {
        // codes: 32 keys of 32 bytes on; 16-bit: 32 bytes of a row
        const int on = C::kCodes ? k * 1024 : (k >> 2) * C::kPBlock + (k & 3) * 32;
        mma(tmem + 2 * C::kN, v + ((k * kStep * C::kPitch) >> 4), pt + (on >> 4),
            id_o, acc || k > 0);
      }
      mma_commit(&bar_free[s]);
      mma_commit(&bar_o[x & 1]);
      return true;
    };
    bool have = next_run(walk, q);
    while (ok && have) {
      ok = mbar_wait(&bar_q, run & 1, w);
      ++run;
      for (int i = 0; ok && i < q.n; ++i, ++g) {
        const unsigned h = 2 * g, s = h % H;
        ok = mbar_wait(&bar_full[s], (h / H) & 1, w);
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = dk0 + ((s * C::kTileBytes) >> 4);
#pragma unroll
        for (int k = 0; k < D / kStep; ++k) {
          const int byte = k * 32, blk = byte / C::kPitch, in = byte % C::kPitch;  // of a row
          mma(tmem + (g & 1) * C::kN, kd + ((blk * C::kBlockBytes + in) >> 4), dq0 + ((blk * C::kQBlock + in) >> 4), id_s,
              k > 0);
        }
        mma_commit(&bar_free[s]);
        mma_commit(&bar_s[g & 1]);
        if (i > 0) ok = add(g - 1, i > 1);
      }
      have = next_run(walk, nx);  // while the softmax works
      if (ok) ok = add(g - 1, q.n > 1);
      q = nx;
    }
    // every MMA issued must be complete before tensor memory is released
    mma_commit(&bar_done);
    mbar_wait_drain(&bar_done, 0, a.wait_limit_ns);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kOwnMmaWarp) tmem_dealloc(tmem, C::kCols);
  // this kernel's end has to mean the end of the pass over the prefix too
  if (threadIdx.x == 0) grid_wait();
}

template <int Kind, int D, int R>
cudaError_t launch_own_r(const ServeArgs& a, bool q_f16, int sms, bool after, cudaStream_t s) {
  using C = OwnCfg<Kind, D, R>;
  static_assert(C::kPerSm == own_per_sm(R, C::kElem, D), "the plan counts the CTAs of an SM that the kernel has");
  OwnParams p;
  p.a = a;
  p.q_f16 = q_f16;
  p.row_groups = (a.group * a.nq + R - 1) / R;
  const uint64_t slabs = (uint64_t)a.B * a.Hk;
  if (!make_map_cache(&p.tk, a.k, C::kElem, D, a.cap, slabs, kBoxKeys) ||
      !make_map_cache(&p.tv, a.v, C::kElem, D, a.cap, slabs, kBoxKeys))
    return note_error("cache tensor map encode", cudaErrorInvalidValue);
  const cudaError_t e = cudaFuncSetAttribute(own_kernel<Kind, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return note_error("cached decoding smem attribute", e);
  return note_error("cached decoding launch", launch_serve_kernel(own_kernel<Kind, D, R>, sms * C::kPerSm, kOwnThreads,
                                                                  C::kSmem, after, s, p));
}

template <int Kind>
cudaError_t launch_own_k(const ServeArgs& a, int D, bool q_f16, int sms, bool after, cudaStream_t s) {
  const int r = own_rows(a.group * a.nq);
  if (D == 64) {
    if (r == 4) return launch_own_r<Kind, 64, 4>(a, q_f16, sms, after, s);
    if (r == 8) return launch_own_r<Kind, 64, 8>(a, q_f16, sms, after, s);
    if (r == 16) return launch_own_r<Kind, 64, 16>(a, q_f16, sms, after, s);
    return launch_own_r<Kind, 64, 24>(a, q_f16, sms, after, s);
  }
  if (r == 4) return launch_own_r<Kind, 128, 4>(a, q_f16, sms, after, s);
  if (r == 8) return launch_own_r<Kind, 128, 8>(a, q_f16, sms, after, s);
  if (r == 16) return launch_own_r<Kind, 128, 16>(a, q_f16, sms, after, s);
  return launch_own_r<Kind, 128, 24>(a, q_f16, sms, after, s);
}

}  // namespace
}  // namespace fa
