// The pass over the shared prefix of a decoding step (fa_decode_shared).
//
// Mathematics.  All B * group * nq query rows that read key head h attend to the
// same np keys, so their scores are one product S = Q K^T of [rows, D] by [D, np]:
// the prefix is read once for the whole batch, and the step is shaped like the
// forward pass (fa_tc_fwd.cu), whose schedule this kernel follows: score tiles
// and accumulators live in tensor memory, a running maximum is rescaled
// lazily, and what leaves the SM is a state (m, l, u) a row for the merge kernel.
//
// Bound.  Up to a few hundred rows a key head, the stream of K and V; beyond, the
// two products.  4 sequences of 64 query heads behind 131072 keys of 8 key heads take 100 us, the stream 79; 256
// sequences of 32 heads behind 32768 of 4, in which a CTA's step takes 1.6 us, 85 % of the tensor rate, 112 on 128 SMs.
//
// Two arrangements of a CTA's two softmax warpgroups ("slots"):
//   pair    rows of a key head > 128: slot t works on query tile 2 pair + t, both on
//           every 128-key tile, so K and V feed two products each;
//   halves  rows <= 128: both slots hold the one query tile, slot t takes keys
//           64 t .. 64 t + 63 of every tile.  A single tile would leave a slot idle and a
//           serial chain product - softmax - product as long as the loads; the halves
//           run side by side and each leaves a state of its own.
//
// Schedule.  A unit is a (key head, query-tile pair); its key tiles are its steps.
// The steps of all units in a row are cut into equal runs, one a CTA, and a
// unit's states are joined over the CTAs that share it.
//
// Hidden keys.  Where a sequence's own part is shorter than its new tokens, causal hides the prefix's
// last keys from some of its rows.  Their weights are zero, but 0 * NaN is not: in the tiles
// that some row does not see whole, the softmax warps put zeros in place of such keys' values that are not finite, and
// the rows that do see them get them at the run's end, as in the pass over the own rows.  One slot does it for both
// where they share the keys (its product is issued first).
//
// Warps and barriers are those of the forward, except that the softmax warps
// write their own Q tile into shared memory (rows of one tile come from many
// sequences) and announce it on bar_q[t], a run's before they read out the last one's state.
#include <math.h>

#include "fa_internal.cuh"
#include "fa_serve.cuh"
#include "fa_tmap.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

using namespace ptx;

constexpr int kBM = kPrefixRows;      // query rows per tile
constexpr int kBN = kPrefixKeys;      // keys per step
constexpr int kThreads = 384;         // 2 softmax warpgroups + 1 support warpgroup
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale when the max grows by > 2^8

struct PrefixParams {
  CUtensorMap tk, tv;
  ServeArgs a;
  PrefixPlan plan;
};

template <int D>
struct Cfg {
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kTileBytes = 128 * D * 2;  // one Q, K or V tile
  static constexpr int kHalves = D / 64;          // 64-column (128-byte) swizzle blocks
  static constexpr int kHalfBytes = 128 * 128;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kSmemBytes = kVOff + kStages * kTileBytes + 1024;
};

template <int D, bool F16, bool kSplit, bool kHide>
__global__ void __launch_bounds__(kThreads, 1) tc_prefix_kernel(const __grid_constant__ PrefixParams p) {
  using C = Cfg<D>;
  constexpr int kCols = kSplit ? kBN / 2 : kBN;  // keys of a slot's score tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // bar_k0: the first K tile; bar_kv[g % stages]: V_g and K_{g+1}.  Steps g are counted
  // over all of the CTA's runs, so rings and per-step barriers keep their phase.  bar_s[t]: an S of
  // slot t (and the P V before it); bar_fin[t]: a run's last P V.  That one has a barrier of its own because
  // the next run's first S may be complete before the softmax looks: two phases of one barrier
  // would pass for none.
  __shared__ __align__(8) uint64_t bar_k0, bar_done;
  __shared__ __align__(8) uint64_t bar_kv[C::kStages], bar_kfree[C::kStages], bar_vfree[C::kStages];
  __shared__ __align__(8) uint64_t bar_q[2], bar_s[2], bar_p[2], bar_fin[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ int s_bad;  // a hidden value was not finite, in this run or an earlier one

  const ServeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = a.group * a.nq;
  const int rows = a.B * gq;  // of a key head
  const int nkt = p.plan.steps;

  // ---- the CTA's runs of steps
  struct Run {
    int hk, row0, j0, n, slots, part;  // slots: 2, or 1 when the pair's second tile has no row
  };
  const long long first = (long long)blockIdx.x * p.plan.per_cta;
  const long long end = min((long long)p.plan.units * nkt, first + p.plan.per_cta);
  auto next_run = [&](long long& t, Run& q) -> bool {
    if (t >= end) return false;
    const int unit = (int)(t / nkt);
    q.j0 = (int)(t - (long long)unit * nkt);
    q.n = (int)min((long long)(nkt - q.j0), end - t);
    q.hk = unit / p.plan.pairs;
    q.row0 = (unit - q.hk * p.plan.pairs) * 2 * kBM;
    q.slots = kSplit || q.row0 + kBM < rows ? 2 : 1;
    q.part = prefix_part(p.plan, unit, blockIdx.x);
    t += q.n;
    return true;
  };

  if (threadIdx.x == 0) {
    mbar_init(&bar_k0, 1);
    mbar_init(&bar_done, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar_kv[s], 1);
      mbar_init(&bar_kfree[s], 1);
      mbar_init(&bar_vfree[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar_q[t], 4);  // one arrival per softmax warp
      mbar_init(&bar_s[t], 1);
      mbar_init(&bar_p[t], 4);
      mbar_init(&bar_fin[t], 1);
    }
    abort_flag = 0;
    s_bad = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // not before the allocation: a kernel started early may take tensor memory too
  grid_launch_dependents();
  const uint32_t tmem = tmem_base_sh;
  const WaitCtx w{&abort_flag, a.status, a.wait_limit_ns};

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<kComputeRegs>();
    const int t = warp >> 2;
    const int quad = warp & 3;          // TMEM lanes 32*quad .. 32*quad+31
    const int r = quad * 32 + lane;     // row within the query tile
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t t_s = tmem + lane_off + t * 128;
    const uint32_t t_o = tmem + lane_off + 256 + t * 128;
    // The prefix keys that row rr of a sequence with len rows of its own sees.
    auto seen = [&](int len, int rr) -> int {
      return a.causal ? (int)max(0ll, min((long long)a.np, (long long)a.np + len - a.nq + rr % a.nq + 1)) : a.np;
    };
    // The keys that all rows of a run's unit see (as far as the run's keys go): what the first new token of every
    // sequence in it sees.
    auto seen_by_all = [&](const Run& q) -> int {
      int lim = a.np;
      if (!kHide || (q.j0 + q.n) * kBN <= a.np - a.nq + 1) return lim;
      const int n = min(rows - q.row0, kSplit ? kBM : 2 * kBM), b0 = q.row0 / gq, b1 = (q.row0 + n - 1) / gq;
      for (int b = b0 + lane; b <= b1; b += 32) {
        const int len = raw_len(a, b);
        if (len_ok(a, len)) lim = min(lim, seen(len, 0));
      }
      return __reduce_min_sync(0xffffffffu, lim);
    };
    // A run's query row to this slot's tile; kmax: the prefix keys that the row sees.
    // Every S of the slot's run before is complete.
    auto put_q = [&](const Run& q, int& kmax) {
      const int row = q.row0 + (kSplit ? 0 : t * kBM) + r;  // row of the key head
      const int b = row / gq, rr = row - b * gq;
      const uint4* src = nullptr;
      kmax = 0;
      int len = -1;
      if (row < rows) {
        len = raw_len(a, b);  // on its way while the queries are read
        src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                             (((long long)b * a.Hk + q.hk) * gq + rr) * D);
      }
      // kLanes lanes read a row together (a row a lane would touch 32 lines an access: 4 us)
      constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
#pragma unroll 1
      for (int i0 = 0; i0 < kLanes; i0 += 8) {  // eight loads in flight; more, or both rounds at once, would spill
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const auto* from = reinterpret_cast<const uint4*>(__shfl_sync(
              0xffffffffu, reinterpret_cast<unsigned long long>(src), (i0 + i) * kAtOnce + lane / kLanes));
          x[i] = from ? __ldg(from + lane % kLanes) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int to = quad * 32 + (i0 + i) * kAtOnce + lane / kLanes, ch = lane % kLanes;  // tile row, 16-byte chunk
          *reinterpret_cast<uint4*>(smem + C::kQOff + t * C::kTileBytes + (ch >> 3) * C::kHalfBytes + to * 128 +
                                    (((ch & 7) ^ (to & 7)) << 4)) = x[i];
        }
      }
      if (len_ok(a, len)) kmax = seen(len, rr);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_q[t]);
    };
    bool ok = true;
    int G = 0;   // steps of the earlier runs
    int cs = 0, fin = 0;  // completions of bar_s[t] and bar_fin[t] seen so far
    long long cur = first;
    Run q, nx;
    int kmax = 0, kmax_next = 0;
    bool have = next_run(cur, q), ready = false;
    // A run's steps and its state.  hide: some row may not see all of its keys (lim_all: those that all see).  Steps that
    // cannot hide any have kernels without it.  Where a slot holds pairs of tiles the loop is there twice, chosen by
    // run: 64 sequences of 20 query rows a key head behind 8192 keys of D 64 take 42.4 us (42.3 without hide; one loop
    // 43.7).  With halved keys one loop is better: 32 of 4 rows behind 4096 keys 73.0 us (72.9 without; two loops 74.6).
    auto work_run = [&](auto hide, int lim_all) {
      const int row = q.row0 + (kSplit ? 0 : t * kBM) + r;
      const bool work = __any_sync(0xffffffffu, kmax > 0);  // a warp without a row only keeps step
      float m_ref = -INFINITY;  // reference maximum of the exponentials (log2 units)
      float l = 0.f;
      for (int j = 0; j < q.n; ++j) {
        const int g = G + j;
        if (!warp_wait(&bar_s[t], cs & 1, w)) {
          ok = false;
          break;
        }
        ++cs;
        if (t == q.slots - 1 && quad == 0 && lane == 0) {
          // S of the last slot is complete, and with it every product issued before
          // it: the other slot's S (K_g is consumed) and both P V of the step before
          mbar_arrive(&bar_kfree[g % C::kStages]);
          if (g > 0) mbar_arrive(&bar_vfree[(g - 1) % C::kStages]);
        }
        tc_fence_after();
        if (work) {
          uint32_t sr[kCols / 32][32];
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) tmem_ld32(t_s + c * 32, sr[c]);
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) tmem_ld_wait(sr[c]);
          const int k0 = (q.j0 + j) * kBN + (kSplit ? t * kCols : 0);
          if (k0 + kCols > kmax) {
            const int cut = kmax - k0;
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c * 32 + e >= cut) sr[c][e] = __float_as_uint(-INFINITY);
          }
          float mp[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) mp[x] = -INFINITY;
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mp[(e >> 1) & 7] =
                  fmax3(mp[(e >> 1) & 7], __uint_as_float(sr[c][e]), __uint_as_float(sr[c][e + 1]));
          const float mt = fmaxf(fmax3(mp[0], mp[1], mp[2]), fmax3(fmax3(mp[3], mp[4], mp[5]), mp[6], mp[7]));
          const float m_new = fmaxf(m_ref, mt * a.c2);
          float alpha = 1.f;
          const bool grow = m_new > m_ref + kRescaleThreshold;
          if (grow) {
            alpha = (m_ref == -INFINITY) ? 0.f : ex2_approx(m_ref - m_new);
            m_ref = m_new;
            l *= alpha;
          }
          const float nmu = (m_ref == -INFINITY) ? 0.f : -m_ref;
          float rs0 = 0.f, rs1 = 0.f;
          // P (16-bit pairs) over the scores, 32 packed columns at a time
#pragma unroll
          for (int hf = 0; hf < kCols / 64; ++hf) {
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int e0 = 64 * hf + 2 * c;
              float a0, a1;
              ffma2(a0, a1, __uint_as_float(sr[e0 >> 5][e0 & 31]), __uint_as_float(sr[(e0 + 1) >> 5][(e0 + 1) & 31]),
                    a.c2, nmu, nmu);
              const float p0 = ex2_approx(a0);
              const float p1 = ex2_approx(a1);
              // The product takes weights of the values' type (its operands have one type), as the forward's does:
              // half a step of it a weight.  The sums take them unrounded.
              fadd2(rs0, rs1, p0, p1);
              pk[c] = pack16x2<F16>(p0, p1);
            }
            tmem_st32(t_s + 32 * hf, pk);
          }
          l += rs0 + rs1;
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            // accumulator rows rescaled in place: the previous P V is complete (the
            // wait on bar_s covers it) and this step's waits for bar_p below
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + c, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(t_o + c, o);
            }
          }
          tmem_st_wait();
        }
        if (hide.value && (q.j0 + j + 1) * kBN > lim_all && (kSplit || t == 0)) {
          // hidden values that are not finite; V_g stays until this slot's warps are in the next step
          if (!warp_wait(&bar_kv[g % C::kStages], (g / C::kStages) & 1, w)) {
            ok = false;
            break;
          }
          // a key a thread; with halved keys two threads share one
          constexpr int kChunks = D / 8 / (kSplit ? 2 : 1);
          const int key = kSplit ? t * kCols + (r & (kCols - 1)) : r, ch0 = kSplit ? r / kCols * kChunks : 0;
          const int at = (q.j0 + j) * kBN + key;
          if (at >= lim_all && at < a.np) {
            uint8_t* v = smem + C::kVOff + (g % C::kStages) * C::kTileBytes + key * 128;
#pragma unroll 1
            for (int c4 = ch0; c4 < ch0 + kChunks; c4 += 4) {
              uint4 u[4];
              auto chunk = [&](int x) {
                return reinterpret_cast<uint4*>(v + ((c4 + x) >> 3) * C::kHalfBytes + ((((c4 + x) & 7) ^ (key & 7)) << 4));
              };
#pragma unroll
              for (int x = 0; x < 4; ++x) u[x] = *chunk(x);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint4 y = make_uint4(finite_only16<F16>(u[x].x), finite_only16<F16>(u[x].y),
                                           finite_only16<F16>(u[x].z), finite_only16<F16>(u[x].w));
                if (u[x].x != y.x || u[x].y != y.y || u[x].z != y.z || u[x].w != y.w) {
                  *chunk(x) = y;
                  *reinterpret_cast<volatile int*>(&s_bad) = 1;
                }
              }
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[t]);
      }
      // the next run's queries, while this one's last product runs: its S is issued
      // after that product, over the weights that it has read by then
      if (ok && have && t < nx.slots) {
        put_q(nx, kmax_next);
        ready = true;
      }
      if (ok && warp_wait(&bar_fin[t], fin & 1, w)) {
        ++fin;
        tc_fence_after();
        // the run's state, in groups of eight columns: a warp's rows are neighbours there
        const long long at = ((long long)q.part * 2 + t) * kBM;
        // the weights' barriers and the product's lie between the last of its writers and here
        const bool bad = hide.value && *reinterpret_cast<volatile int*>(&s_bad) != 0;
        if (work) {
          float* u = a.pre_u + at * D + r * 8;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + c, o);
            tmem_ld_wait(o);
            if (bad) {  // hidden from other rows, not from this one
              const int k1 = min(kmax, (q.j0 + q.n) * kBN);
#pragma unroll 1
              for (int key = max(lim_all, q.j0 * kBN); key < k1; ++key) {
                if (kSplit && ((key / kCols) & 1) != t) continue;  // the other slot's
                const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.vp) +
                                                                   ((long long)q.hk * a.np + key) * D + c);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const uint4 y = __ldg(from + x);
                  const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t not_finite = yw[e] ^ finite_only16<F16>(yw[e]);  // the others: +0
                    float2 f;
                    if constexpr (F16)
                      f = __half22float2(*reinterpret_cast<const __half2*>(&not_finite));
                    else
                      f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&not_finite));
                    uint32_t& o0 = o[8 * x + 2 * e];
                    uint32_t& o1 = o[8 * x + 2 * e + 1];
                    o0 = __float_as_uint(__uint_as_float(o0) + f.x);
                    o1 = __float_as_uint(__uint_as_float(o1) + f.y);
                  }
                }
              }
            }
            if (row < rows)
#pragma unroll
              for (int x = 0; x < 32; x += 8) store32(u + ((c + x) >> 3) * (kBM * 8), o + x);
          }
        }
        if (row < rows) a.pre_ml[at + r] = make_float4(m_ref, l, work ? m_ref : -INFINITY, 0.f);
      } else {
        ok = false;
      }
    };
    while (ok && have) {
      have = next_run(cur, nx);
      if (t < q.slots) {
        if (ready)
          kmax = kmax_next;
        else
          put_q(q, kmax);
        ready = false;
        const int lim_all = seen_by_all(q);
        if constexpr (kHide && !kSplit) {
          if (lim_all < a.np)
            work_run(Flag<true>{}, lim_all);
          else
            work_run(Flag<false>{}, lim_all);
        } else {
          work_run(Flag<kHide>{}, lim_all);
        }
      }
      G += q.n;
      q = nx;
    }
  } else {
    // warps 8-11: producer, MMA issuer and two idle warps completing the warpgroup
    setmaxnreg_dec<kSupportRegs>();
    if (warp == kTmaWarp && lane == 0) {
      // ---------------------------------------------------------- producer
      tma_prefetch_desc(&p.tk);
      tma_prefetch_desc(&p.tv);
      auto load = [&](int off, const CUtensorMap* map, const Run& q, int j, int g, uint64_t* bar) {
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(smem + off + (g % C::kStages) * C::kTileBytes + hf * C::kHalfBytes, map, bar, hf * 64,
                      (q.j0 + j) * kBN, q.hk);
      };
      // Stage release as in the forward: V_g and K_{g+1} both need the release of step
      // g + 1 - stages and share one barrier.
      int issued = 0, G = 0;
      bool good = true;
      long long cur = first;
      Run q, nx;
      if (next_run(cur, q)) {
        mbar_arrive_expect_tx(&bar_k0, C::kTileBytes);
        load(C::kKOff, &p.tk, q, 0, 0, &bar_k0);
        bool have = true;
        while (good && have) {
          const bool has_next = next_run(cur, nx);
          for (int j = 0; j < q.n; ++j) {
            const int g = G + j;
            const int s = g % C::kStages;
            const bool k_next = j + 1 < q.n || has_next;
            if (g >= C::kStages && !mbar_wait(&bar_vfree[s], (g / C::kStages - 1) & 1, w)) {
              good = false;
              break;
            }
            if (k_next && g + 1 >= C::kStages &&
                !mbar_wait(&bar_kfree[(g + 1) % C::kStages], ((g + 1) / C::kStages - 1) & 1, w)) {
              good = false;
              break;
            }
            mbar_arrive_expect_tx(&bar_kv[s], (k_next ? 2 : 1) * C::kTileBytes);
            load(C::kVOff, &p.tv, q, j, g, &bar_kv[s]);
            if (k_next) {
              if (j + 1 < q.n)
                load(C::kKOff, &p.tk, q, j + 1, g + 1, &bar_kv[s]);
              else
                load(C::kKOff, &p.tk, nx, 0, g + 1, &bar_kv[s]);
            }
            issued = g + 1;
          }
          G += q.n;
          q = nx;
          have = has_next;
        }
        if (abort_flag) {
          // let copies already in flight land before the CTA's memory is released
          mbar_wait_drain(&bar_k0, 0, a.wait_limit_ns);
          for (int g = max(0, issued - C::kStages); g < issued; ++g)
            mbar_wait_drain(&bar_kv[g % C::kStages], (g / C::kStages) & 1, a.wait_limit_ns);
        }
      }
    } else if (warp == kMmaWarp && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t id_s = idesc16<F16>(kBM, kCols, false, false);
      const uint32_t id_o = idesc16<F16>(kBM, D, false, true);
      const uint64_t dq0 = sdesc_sw128(smem_u32(smem + C::kQOff), 16, 1024);
      const uint64_t dk0 = sdesc_sw128(smem_u32(smem + C::kKOff), 16, 1024);
      const uint64_t dv0 = sdesc_sw128(smem_u32(smem + C::kVOff), C::kHalfBytes, 1024);
      constexpr uint32_t kSlotKeys = kSplit ? (kCols * 128) >> 4 : 0;  // slot 1's keys within a tile
      // S_t = Q_t K^T (both K-major): D/16 MMAs of K = 16, issued back to back
      auto issue_s = [&](int t, int s) {
        const uint64_t a0 = dq0 + ((t * C::kTileBytes) >> 4);
        const uint64_t b0 = dk0 + ((s * C::kTileBytes) >> 4) + t * kSlotKeys;
        if constexpr (D == 128) {
          uint64_t x[8], y[8];
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t off = ((ks >> 2) * C::kHalfBytes + (ks & 3) * 32) >> 4;
            x[ks] = a0 + off;
            y[ks] = b0 + off;
          }
          mma_ss_x8(tmem + t * 128, x, y, id_s, 0u);
        } else {
          uint64_t x[4], y[4];
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            x[ks] = a0 + ks * 2;
            y[ks] = b0 + ks * 2;
          }
          mma_ss_x4(tmem + t * 128, x, y, id_s, 0u);
        }
      };
      // O_t += P_t V (P from TMEM, V MN-major): MMAs of K = 16 keys
      auto issue_pv = [&](int t, int s, bool acc) {
        const uint64_t b0 = dv0 + ((s * C::kTileBytes) >> 4) + t * kSlotKeys;
        uint32_t x[kCols / 16];
        uint64_t y[kCols / 16];
#pragma unroll
        for (int ks = 0; ks < kCols / 16; ++ks) {
          x[ks] = tmem + t * 128 + ks * 8;
          y[ks] = b0 + ((ks * 2048) >> 4);
        }
        if constexpr (kSplit)
          mma_ts_x4(tmem + 256 + t * 128, x, y, id_o, acc ? 1u : 0u);
        else
          mma_ts_x8(tmem + 256 + t * 128, x, y, id_o, acc ? 1u : 0u);
      };
      bool ok = true;
      int G = 0;
      int cp[2] = {0, 0};    // completions of bar_p[t] waited for
      int used[2] = {0, 0};  // runs that used slot t so far
      long long cur = first;
      Run q;
      if (end > first) ok = mbar_wait(&bar_k0, 0, w);
      while (ok && next_run(cur, q)) {
        // a later run's first K came with the previous run's last V, which was waited
        // for; each slot's S goes over columns its softmax warps have finished with
        for (int t = 0; t < q.slots; ++t) {
          if (!mbar_wait(&bar_q[t], used[t] & 1, w)) {
            ok = false;
            break;
          }
          ++used[t];
          tc_fence_after();
          issue_s(t, G % C::kStages);
          mma_commit(&bar_s[t]);
        }
        for (int j = 0; ok && j < q.n; ++j) {
          const int g = G + j;
          const int s = g % C::kStages, s1 = (g + 1) % C::kStages;
          if (!mbar_wait(&bar_kv[s], (g / C::kStages) & 1, w)) {  // V_g and K_{g+1}
            ok = false;
            break;
          }
          tc_fence_after();
          for (int t = 0; t < q.slots; ++t) {
            if (!mbar_wait(&bar_p[t], cp[t] & 1, w)) {
              ok = false;
              break;
            }
            ++cp[t];
            tc_fence_after();
            issue_pv(t, s, j > 0);
            if (j + 1 < q.n) issue_s(t, s1);
            mma_commit(j + 1 < q.n ? &bar_s[t] : &bar_fin[t]);
          }
        }
        G += q.n;
      }
      // every MMA issued must be complete before tensor memory is released
      mma_commit(&bar_done);
      mbar_wait_drain(&bar_done, 0, a.wait_limit_ns);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D, bool F16, bool kSplit, bool kHide>
cudaError_t launch_prefix_d(const ServeArgs& a, const PrefixPlan& plan, cudaStream_t s) {
  using C = Cfg<D>;
  PrefixParams p;
  p.a = a;
  p.plan = plan;
  if (!make_map_cache(&p.tk, a.kp, 2, D, a.np, a.Hk, kBN) || !make_map_cache(&p.tv, a.vp, 2, D, a.np, a.Hk, kBN))
    return note_error("prefix tensor map encode", cudaErrorInvalidValue);
  const cudaError_t e = cudaFuncSetAttribute(tc_prefix_kernel<D, F16, kSplit, kHide>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return note_error("prefix smem attribute", e);
  return note_error("prefix launch", launch_serve_kernel(tc_prefix_kernel<D, F16, kSplit, kHide>, plan.ctas, kThreads,
                                                         C::kSmemBytes, false, s, p));
}

template <int D, bool F16, bool kHide>
cudaError_t launch_prefix_h(const ServeArgs& a, const PrefixPlan& plan, cudaStream_t s) {
  return plan.split ? launch_prefix_d<D, F16, true, kHide>(a, plan, s) : launch_prefix_d<D, F16, false, kHide>(a, plan, s);
}

// One new token is the last of its sequence, and sees the whole prefix.
template <int D, bool F16>
cudaError_t launch_prefix_f(const ServeArgs& a, const PrefixPlan& plan, cudaStream_t s) {
  return a.causal && a.nq > 1 ? launch_prefix_h<D, F16, true>(a, plan, s) : launch_prefix_h<D, F16, false>(a, plan, s);
}

}  // namespace

cudaError_t launch_prefix(const ServeArgs& a, const PrefixPlan& plan, int D, bool f16, cudaStream_t s) {
  if (D == 64) return f16 ? launch_prefix_f<64, true>(a, plan, s) : launch_prefix_f<64, false>(a, plan, s);
  return f16 ? launch_prefix_f<128, true>(a, plan, s) : launch_prefix_f<128, false>(a, plan, s);
}

}  // namespace fa
