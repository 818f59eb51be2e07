// What the kernels of a decoding step over a cache share: how the work is cut,
// and where the states of the pieces lie in the workspace.
//
// A state of a query row over some keys is (m, l, mu, u): the weights' sum is
// l 2^m and the weighted value sum u 2^mu (log2 units).
#pragma once

#include <math.h>

#include "fa_internal.cuh"

namespace fa {

// SMs the work is cut for.  Nothing depends on how many there are or on what runs at
// once, and the workspace's size must not depend on the device.
constexpr int kSms = 152;
// The pass over the own rows (fa_serve_own.cuh): at most two CTAs an SM.
constexpr int kOwnCtas = 2 * kSms;
constexpr int kOwnTile = 128;  // keys of a step
// What a run costs besides its tiles (queries in, references found, state out), in tiles: it
// only steers the cut.  About as long as 96 KB of cache take, 160 KB at 24 rows: fitted over the CTAs of
// ragged batches, 3 and 5 tiles of 32 KB (8-bit, D = 128), below one of 64 KB (16-bit).  Without it the CTAs that got
// the short sequences took twice the average; 24 rows of 24 sequences of up to 16384 keys took 88 us with 3, 84 with 5.
inline int own_run_cost(int cta_rows, int elem_bytes, int D) {
  return (cta_rows == 24 ? 160 : 96) * 1024 / (2 * kOwnTile * D * elem_bytes);
}
// Query rows of a CTA: what the rows of a key head fill, so that fewer rows leave fewer
// columns to multiply and read out.  More than 24 are spread over row groups, which
// read the same keys at about the same time, so mostly from L2.
inline int own_rows(int rows) {
  if (rows <= 16) return rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
  return (rows + 15) / 16 <= (rows + 23) / 24 ? 16 : 24;  // the fewest groups, then the fewest rows
}
// CTAs of an SM: two, but where their rings of tiles leave no room for a second (OwnCfg checks it).
constexpr int own_per_sm(int cta_rows, int elem_bytes, int D) {
  return cta_rows == 24 && elem_bytes == 2 && D == 128 ? 1 : 2;
}

// A length out of range counts as 0 (reported here and by the join, which leaves its rows alone).
__device__ __forceinline__ int raw_len(const ServeArgs& a, int b) { return a.lens ? __ldg(a.lens + b) : a.max_len; }
__device__ __forceinline__ bool len_ok(const ServeArgs& a, int len) { return len >= 0 && len <= a.max_len; }
__device__ __forceinline__ int seq_len(const ServeArgs& a, int b) {
  const int len = raw_len(a, b);
  return len_ok(a, len) ? len : 0;
}
__host__ __device__ __forceinline__ int own_tiles(int len) { return (int)(((unsigned)len + kOwnTile - 1) / kOwnTile); }
// Cost of a unit of `tiles` tiles: the run's own cost, then a tile each.
__device__ __forceinline__ int own_cost(const ServeArgs& a, int tiles) { return tiles > 0 ? tiles + a.run_cost : 0; }

// A truth value that a generic lambda can take as a type.
template <bool B>
struct Flag {
  static constexpr bool value = B;
};

// Elements of a word of two 16-bit values that are not finite become zero.
template <bool F16>
__device__ __forceinline__ uint32_t finite_only16(uint32_t w) {
  constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (((w >> (16 * i)) & kExp) == kExp) w &= ~(0xffffu << (16 * i));
  return w;
}

// Factor of a state with maximum m joined under the maximum mm >= m: 1 for
// equal maxima, -inf among them (that state holds nothing, or only NaN).
__device__ __forceinline__ float join_factor(float m, float mm) { return m == mm ? 1.f : exp2f(m - mm); }

// A CTA's share [first, end) of the cost of all sequences laid out in a row
// (sequence-major, units -- key head, row group -- of a sequence, in a unit the run's own cost and then its
// tiles).  Position `first` is `off` into unit (b, hk, rg).  A tile belongs to the CTA
// whose share its position falls into.
struct OwnPlan {
  long long first, end;
  int b, hk, rg, off;
};

// Works out the CTA's share.  Block-wide; the caller's shared memory may be
// initialised before it, since it ends with a block-wide barrier.  CTA 0 also
// leaves the layout for the merge kernel: a.plan[0] = a CTA's share, a.plan[1 + b] = what
// lies before sequence b.
template <int kThreads>
__device__ __forceinline__ void own_plan(const ServeArgs& a, int row_groups, OwnPlan& plan) {
  __shared__ long long s_sum[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long units = (long long)a.Hk * row_groups;  // of one sequence
  auto cost = [&](int b) -> long long {
    if (b >= a.B) return 0;
    const int len = raw_len(a, b);
    if (!len_ok(a, len)) {
      if (blockIdx.x == 0) atomicOr(a.status, kDevBadSeqlens);
      return 0;
    }
    return (long long)own_cost(a, own_tiles(len)) * units;
  };
  const long long mine = cost(threadIdx.x);  // the first kThreads sequences: enough for most batches
  long long x = mine;
  for (int b = threadIdx.x + kThreads; b < a.B; b += kThreads) x += cost(b);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  if (lane == 0) s_sum[warp] = x;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) total += s_sum[i];
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long first = min(total, per * blockIdx.x);
  if (threadIdx.x == 0) {
    plan.first = first;
    plan.end = min(total, first + per);
    if (blockIdx.x == 0) a.plan[0] = per;
  }
  long long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const long long n = b0 == 0 ? mine : cost(b);
    long long incl = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += y;
    }
    __syncthreads();  // the last reads of s_sum
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    long long at = before + incl - n;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) at += s_sum[i];
      before += s_sum[i];
    }
    if (b < a.B && at <= first && first < at + n) {
      const long long unit_cost = n / units, unit = (first - at) / unit_cost;
      plan.b = b;
      plan.hk = (int)(unit / row_groups);
      plan.rg = (int)(unit - (long long)plan.hk * row_groups);
      plan.off = (int)(first - at - unit * unit_cost);
    }
    if (blockIdx.x == 0 && b < a.B) a.plan[1 + b] = at;
  }
  __syncthreads();
}

// Where a run's state goes: whole units to their rows' place, a unit's cut ends
// to one of two places of the CTA (one for the part that continues a unit, one
// for the part that begins it).
struct PartSlot {
  float* u;
  float4* ml;  // (m, l, mu, unused)
};
__device__ __forceinline__ PartSlot own_slot(const ServeArgs& a, int cta, bool begins, bool ends, long long row,
                                             int cta_rows, int D) {
  if (begins && ends) return PartSlot{a.row_u + row * D, a.row_ml + row};
  const long long r = ((long long)cta * 2 + (begins ? 1 : 0)) * cta_rows;
  return PartSlot{a.cut_u + r * D, a.cut_ml + r};
}

// The pass over the prefix (fa_tc_prefix.cu): units of kPrefixRows (split) or
// 2 kPrefixRows query rows of a key head, each of `steps` tiles of kPrefixKeys keys;
// all units' steps in a row, per_cta of them a CTA, a CTA an SM.
constexpr int kPrefixRows = 128, kPrefixKeys = 128;
struct PrefixPlan {
  int split;              // at most kPrefixRows rows: the two slots share them and halve the keys
  int pairs, steps, units;
  int ctas, parts;        // parts: states kept for a unit (CTAs that may share it)
  long long per_cta;
};
// `per` steps a CTA, or as few as that many CTAs need.
inline PrefixPlan prefix_plan_of(PrefixPlan p, long long per) {
  const long long all = (long long)p.units * p.steps;
  p.ctas = (int)((all + per - 1) / per);
  p.per_cta = (all + p.ctas - 1) / p.ctas;
  p.ctas = (int)((all + p.per_cta - 1) / p.per_cta);
  p.parts = (int)((p.steps - 1) / p.per_cta) + 2;
  return p;
}
// On `ctas` CTAs at most.
inline PrefixPlan prefix_plan(int B, int Hk, int gq, int np, int ctas) {
  PrefixPlan p = {};
  const long long rows = (long long)B * gq;
  p.split = rows <= kPrefixRows;
  p.pairs = (int)((rows + 2 * kPrefixRows - 1) / (2 * kPrefixRows));
  p.steps = (np + kPrefixKeys - 1) / kPrefixKeys;
  p.units = p.pairs * Hk;
  const long long all = (long long)p.units * p.steps;
  return all > 0 ? prefix_plan_of(p, (all + ctas - 1) / ctas) : p;
}

// How a step is laid over the SMs.  With a prefix and own rows, the two passes run
// side by side, the prefix on as many SMs as let both end at about the same time: each pass's
// start and end (its queries, first copies, states) hides behind the other's stream.  64 sequences behind 8192 keys,
// 16-bit rows of up to 1024: 60 us one after the other, 46 side by side on 52 + 100 SMs (50 on 43 + 109 or 76 + 76);
// 4 drafted tokens of 32 behind 4096, 8-bit rows of up to 2048: 94, and 73 on 32 + 120 (98 on 24 + 128, 79 on 57 + 95); 256
// behind 32768: 134, and 120 on 128 + 24 (132 on 124 + 28, 126 on 132 + 20).
// The lengths are on the device, so the own rows are taken to be a little over half of max_len, the mean of
// lengths spread evenly below it.  That is a guess, and max_len the caller's means to better it: shorter rows end
// early and leave the rest to the prefix's few SMs.  Up to 200 16-bit rows of 64 sequences behind 8192 keys: 30 us with max_len
// 200, 36 with 1024, 80 with 4096, 132 with 8192, 420 with 32768 (8-bit rows: 29, 40, 51, 63, 214).
// The workspace's size and the launch have to get the same plan: one copy of the arithmetic, never inlined.
struct ServePlan {
  PrefixPlan pre;
  int own_sms;
  bool together;  // the prefix goes first, and the own rows start on the SMs that it leaves
};
__noinline__ inline ServePlan serve_plan(int B, int Hk, int gq, int np, int max_len, int D, int elem_bytes) {
  ServePlan s;
  s.together = np > 0 && max_len > 0;
  s.pre = prefix_plan(B, Hk, gq, np, kSms);
  s.own_sms = kSms;
  if (!s.together) return s;
  // Times in us, fitted to the CTAs of those and other batches.  Own rows on m SMs, own_per_sm CTAs an SM: 6 to begin, a
  // tile 1.1 (16 rows 1.2, 24 rows 1.5), a run 3 (16-bit 1, 24 rows 5), and no less than the stream at 6.5 TB/s.  Tiles of 64 KB
  // (D = 128 in 16 bits) 1.7 (4096 of them on 15, 30, 50 SMs: 241, 128, 84 us at 4 rows, 256, 135, 89 at 16); where a CTA has its
  // SM to itself 1.2 alone (343, 180, 114 at 20 rows), 1.5 beside a prefix, a run 3.  (Two CTAs counted where there is one: 8
  // sequences of 5 new tokens, 8 key heads, 65536 + up to 2048 16-bit keys took 131 us on 142 + 10 SMs, 75 on 128 + 24.)
  const int rows = own_rows(gq), per_sm = own_per_sm(rows, elem_bytes, D);
  const double units = (double)B * Hk * ((gq + rows - 1) / rows), tiles = units * (0.55 * max_len / kOwnTile + 0.5);
  const double tile_us = D * elem_bytes == 256 ? (per_sm == 1 ? 1.5 : 1.7) : rows <= 8 ? 1.1 : rows == 16 ? 1.2 : 1.5;
  const double run_us = per_sm == 1 ? 3.0 : rows == 24 ? 5.0 : elem_bytes == 1 ? 3.0 : 1.0;
  const double stream = 6 + tiles * (2.0 * kOwnTile * D * elem_bytes) / 6.5e6;
  const double own0 = 6 + run_us, own = (tiles * tile_us + units * run_us) / per_sm;
  // The prefix on n SMs: 9 at its ends, a step 1.7 with halved keys, else 1.6, or 2.2 beside a stream that takes the
  // memory's rate, and 2.5 for every further unit that a CTA touches (64 sequences of 5 new tokens behind 1024 keys, 40
  // units of 8 steps: 59 us at 20 steps a CTA, 75 at 27, 95 at 40, 141 at 64).
  // And the join 0.25 a state (4 sequences of 24 query rows a key head behind 5000 keys: 23 us with 20 states a row, 26 with 40, 36 with 80).
  constexpr double kUnitUs = 2.5, kStateUs = 0.25;
  const double step_us = (s.pre.split ? 1.7 : stream - 6 > own / kSms ? 2.2 : 1.6) * (D == 128 ? 1.0 : 0.65);
  const double steps = (double)s.pre.units * s.pre.steps, pre = steps * step_us + s.pre.units * kUnitUs;
  // own0 + own / (kSms - n) = 9 + pre / n
  const double d = own0 - 9, b = d * kSms + own + pre;
  double n = 2 * pre * kSms / (b + sqrt(b * b - 4 * d * pre * kSms));
  if (own0 + own / (kSms - n) < stream && stream > 9 + pre / n) n = pre / (stream - 9);
  // The CTAs take whole steps: of the two whole n beside it and the cuts nearest to them that fall on the units' ends
  // or divide the units evenly, the one whose longer pass is the shortest (5 sequences of 8 new tokens, 30 key heads, 28414 + up
  // to 183 keys: 100 us on 148 + 4 SMs, 89 on 145 + 7; 2 sequences of 8 new tokens and 7 key heads, units of 10 steps: 22.4 us
  // with 3 steps a CTA, 18.5 with 2; 61 of 5, units of 7: 26.5 with 6, 23.9 with 7).
  double best = -1;
  auto weigh = [&](long long per) {
    const PrefixPlan plan = prefix_plan_of(s.pre, per);
    if (plan.ctas > kSms - 4) return;
    const long long n_steps = plan.steps, p = plan.per_cta;
    const long long further = n_steps % p == 0 ? 0 : p % n_steps == 0 ? p / n_steps - 1 : (p + n_steps - 2) / n_steps;
    const double join = kStateUs * (n_steps / p) * (plan.split ? 2 : 1);
    const double us = fmax(fmax(own0 + own / (kSms - plan.ctas), stream), 9 + p * step_us + further * kUnitUs) + join;
    if (best < 0 || us < best) {
      best = us;
      s.pre = plan;
    }
  };
  const long long all = (long long)s.pre.units * s.pre.steps, n_steps = s.pre.steps;
  const long long few = n < 1 ? 1 : n > kSms - 5 ? kSms - 5 : (long long)n;
  const long long high = (all + few - 1) / few, low = (all + few) / (few + 1);  // steps a CTA
  weigh(high);
  weigh(low);
  if (low >= n_steps) {
    weigh(low / n_steps * n_steps);
    weigh((high + n_steps - 1) / n_steps * n_steps);
  } else {
    for (long long k = 1; k <= 16 && low - k > 0; ++k)
      if (n_steps % (low - k) == 0) {
        weigh(low - k);
        break;
      }
    for (long long k = 1; k <= 16 && high + k <= n_steps; ++k)
      if (n_steps % (high + k) == 0) {
        weigh(high + k);
        break;
      }
  }
  s.own_sms = kSms - s.pre.ctas;
  return s;
}
// The state's place of a unit's part that CTA `cta` works on.
__device__ __forceinline__ int prefix_part(const PrefixPlan& p, int unit, int cta) {
  return unit * p.parts + (cta - (int)((long long)unit * p.steps / p.per_cta));
}

// Launches a kernel that takes its parameters by value; `after`: it may start
// before the kernel in front of it has finished (and waits for it with
// grid_wait where it needs its results).
template <typename P>
cudaError_t launch_serve_kernel(void (*kernel)(P), int ctas, int threads, int smem, bool after, cudaStream_t s,
                                const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  note_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace fa
