// Column sums of the softmax weights on the tensor cores (bf16 configurations), the second half of
// zha_dense_weights: acc_out[h][k] = acc_in[h][k] + sum over rows r of 2^(c q_r.k - lse_r).
//
// The products are computed again with keys as the rows: S^T = K Q^T, 128 keys x 128 query rows per
// product, so that a column sum is one thread's sum over its own accumulator row
// and no exchange between threads is needed.  Two streams of 128 keys share every
// tile of query rows; each has two accumulators in tensor memory, so that one tile's product runs under the other's
// exponentials, and two warpgroups, each for half of a tile's columns: with one warpgroup the exponential unit stood
// still between tiles for a quarter of the time, with two on alternate tiles both accumulators came free at the same
// time and the products had nothing to run under (64 queries x 8 heads over 64K tokens, the whole call: 129, 116 and
// 114 us).  The two warpgroups of a stream add up at a segment's end.
// Per tile and stream 512 cycles of products (d = 128) against 1024 of exponentials (16 per cycle and SM): the
// exponentials bound it (the unit is busy 65 % of the time), for few row tiles the second read of K.  Taking part of
// the exponentials to the FMA pipe by a polynomial was slower (132 -> 142 us): the issue slots are needed.
//
// Work split: a segment is 256 keys of one KV head against the row tiles that see
// them; all row tiles of all segments form one flat list that is cut evenly over
// the CTAs.  A segment inside one CTA is written out directly, one cut by
// a CTA border leaves partial sums that weights_tc_join_kernel adds in CTA order.
//
// Roles: warps 0-15 the keys (warpgroup g: stream g & 1, columns 64 (g >> 1) on), warp 16 the loads (K pairs, row
// tiles), warp 17 the products, warp 18 the row tiles' log-sum-exps.
#include <cstring>

#include "zha_rows.cuh"
#include "zha_tc.cuh"

namespace zha {

constexpr int kWtThreads = 608;
constexpr int kWtKeys = 256;   // keys per segment
constexpr int kWtCols = 128;   // query rows per tile (columns of the product)
constexpr int kWtSlots = 2;    // row tiles in flight
constexpr int kWtLse = 4;      // tiles whose log-sum-exps are in shared memory (they stay until the tile has been added)
constexpr int kWtFloats = 148 * 2 * kWtKeys;  // partial sums: two slots per CTA

template <int D> struct WtShape {
  static constexpr int kHalf = 128 * D * 2;                 // bytes of 128 keys, or of a row tile
  static constexpr int kSmem = 2 * 2 * kHalf + kWtSlots * kHalf + 1024;
};

// Geometry of the flat list.  Up to 128 query heads of one KV head: a tile is `tok` whole tokens; more: 128 heads
// of one token.
struct WtPlan {
  int tok, per_tok;  // tokens per tile, or tiles per token
  int tiles;         // row tiles of all m tokens
  int segs, full;    // segments per head; of these, the first `full` are seen by every row
  int head;          // list length of one head
  Shares sh;
};

__device__ __forceinline__ int wt_first_tile(const WeightsArgs& a, const WtPlan& p, int seg) {
  if (!a.causal) return 0;
  const int tok = int(max64(0, int64_t(seg) * kWtKeys - (a.n - a.m)));  // first token that sees the segment's first key
  return p.tok > 0 ? tok / p.tok : tok * p.per_tok;
}

__device__ __forceinline__ WtPlan wt_plan(const WeightsArgs& a, int nc) {
  WtPlan p;
  p.tok = a.group <= kWtCols ? kWtCols / a.group : 0;
  p.per_tok = a.group <= kWtCols ? 1 : (a.group + kWtCols - 1) / kWtCols;
  p.tiles = p.tok > 0 ? (a.m + p.tok - 1) / p.tok : a.m * p.per_tok;
  p.segs = int((a.n + kWtKeys - 1) / kWtKeys);
  p.full = a.causal ? min(p.segs, int((a.n - a.m) / kWtKeys) + 1) : p.segs;
  p.head = p.full * p.tiles + warp_total(p.segs - p.full, [&](int i) { return p.tiles - wt_first_tile(a, p, p.full + i); });
  p.sh.set(p.head * a.hkv, nc);
  return p;
}

struct WtSeg {
  int h, seg;
  int first, tiles;  // place in the list and number of its tiles
  int t_first;       // its first row tile
};

__device__ __forceinline__ WtSeg wt_find(const WeightsArgs& a, const WtPlan& p, int x) {
  WtSeg s;
  s.h = x / p.head;
  const int r = x - s.h * p.head;
  int base;
  if (r < p.full * p.tiles) {
    s.seg = r / p.tiles;
    base = s.seg * p.tiles;
  } else {
    const int i = warp_find(p.segs - p.full, [&](int q) { return p.tiles - wt_first_tile(a, p, p.full + q); },
                            r - p.full * p.tiles, &base);
    s.seg = p.full + i;
    base += p.full * p.tiles;
  }
  s.t_first = wt_first_tile(a, p, s.seg);
  s.tiles = p.tiles - s.t_first;
  s.first = s.h * p.head + base;
  return s;
}

// Tokens, heads and number of rows of row tile t: column c is token tok0 + c / gw, head g0 + c % gw.
struct WtTile {
  int tok0, g0, gw, cols;
};
__device__ __forceinline__ WtTile wt_tile(const WeightsArgs& a, const WtPlan& p, int t) {
  WtTile w;
  if (p.tok > 0) {
    w.tok0 = t * p.tok;
    w.g0 = 0;
    w.gw = a.group;
    w.cols = min(p.tok, a.m - w.tok0) * a.group;
  } else {
    w.tok0 = t / p.per_tok;
    w.g0 = (t - w.tok0 * p.per_tok) * kWtCols;
    w.gw = kWtCols;
    w.cols = a.group - w.g0 < kWtCols ? a.group - w.g0 : kWtCols;
  }
  return w;
}

// Rows that one copy of a row tile writes.
__device__ __forceinline__ int wt_box_rows(int group) { return group <= kWtCols ? kWtCols / group * group : kWtCols; }

struct WtMaps {
  CUtensorMap k, q;
};

template <int D>
__global__ void __launch_bounds__(kWtThreads, 1) weights_tc_kernel(WeightsArgs a, const __grid_constant__ WtMaps maps) {
  using Sh = WtShape<D>;
  constexpr int NS = kWtSlots, NL = kWtLse, PANELS = D / 64;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * NS + 21 + 2 * NL];
  __shared__ float other[2][2][128];  // [segment parity][stream]: sums of the stream's second warpgroup
  __shared__ __align__(16) float minus_lse[NL][kWtCols];  // in powers of two; -inf where a tile has no row
  __shared__ uint32_t tmem_base;
  __shared__ Waits waits;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t k_sm = base, ring = base + 4 * Sh::kHalf;  // K: [pair slot][stream]
  const uint32_t b0 = smem_u32(bars);
  auto full = [&](int s) { return b0 + 8 * s; };
  auto empty = [&](int s) { return b0 + 8 * (NS + s); };
  auto k_full = [&](int s) { return b0 + 8 * (2 * NS + s); };
  auto k_empty = [&](int s) { return b0 + 8 * (2 * NS + 2 + s); };
  auto s_full = [&](int st, int b) { return b0 + 8 * (2 * NS + 4 + 2 * st + b); };
  auto s_free = [&](int st, int b) { return b0 + 8 * (2 * NS + 8 + 2 * st + b); };
  const uint32_t done = b0 + 8 * (2 * NS + 12);
  auto x_full = [&](int par, int st) { return done + 8 + 8 * (2 * par + st); };
  auto l_full = [&](int s) { return done + 72 + 8 * s; };
  auto l_empty = [&](int s) { return done + 72 + 8 * (NL + s); };
  auto x_free = [&](int par, int st) { return done + 40 + 8 * (2 * par + st); };
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      bar_init(full(s), 1);
      bar_init(empty(s), 1);
    }
    for (int s = 0; s < NL; ++s) {
      bar_init(l_full(s), 1);
      bar_init(l_empty(s), 16);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(k_full(s), 1);
      bar_init(k_empty(s), 1);
      for (int b = 0; b < 2; ++b) {
        bar_init(s_full(s, b), 1);
        bar_init(s_free(s, b), 8);
        bar_init(x_full(b, s), 4);
        bar_init(x_free(b, s), 4);
      }
    }
    bar_init(done, 1);
    waits.gave_up = 0;
    waits.limit = a.wait_limit;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // rows of a tile that no copy writes (heads that do not divide 128) stay zero
  for (int i = tid; i < NS * Sh::kHalf / 16; i += kWtThreads)
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(ring + i * 16), "r"(0) : "memory");
  fence_async_smem();
  if (wid == 17) tmem_alloc(smem_u32(&tmem_base), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  pdl_trigger();
  pdl_wait();
  const WtPlan plan = wt_plan(a, gridDim.x);
  const int x_begin = plan.sh.begin(blockIdx.x), x_end = plan.sh.begin(blockIdx.x + 1);
  int x = x_begin;

  if (wid == 16) {  // ---------------------------------------------------------------- loads
    int slot = 0, ks = 0;
    uint32_t round = 0, k_round = 0;
    bool ok = true;
    const uint64_t many = l2_evict_normal();
    const uint32_t tile_bytes = uint32_t(wt_box_rows(a.group)) * D * 2;
    while (x < x_end && ok) {
      const WtSeg s = wt_find(a, plan, x);
      const int t1 = min(s.first + s.tiles, x_end) - s.first;
      if (!(ok = bar_wait(k_empty(ks), (k_round & 1) ^ 1, &waits))) break;
      if (lane == 0) {
        bar_expect(k_full(ks), 2 * Sh::kHalf);
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int p = 0; p < PANELS; ++p)
            tma_load(k_sm + (2 * ks + st) * Sh::kHalf + p * 128 * 128, &maps.k, k_full(ks), p * 64,
                     s.seg * kWtKeys + st * 128, s.h, many);
      }
      if (++ks == 2) {
        ks = 0;
        ++k_round;
      }
      for (int t = x - s.first; t < t1; ++t) {
        const WtTile w = wt_tile(a, plan, s.t_first + t);
        if (!(ok = bar_wait(empty(slot), (round & 1) ^ 1, &waits))) break;
        if (lane == 0) {
          bar_expect(full(slot), tile_bytes);
#pragma unroll
          for (int p = 0; p < PANELS; ++p)
            tma_load(ring + slot * Sh::kHalf + p * 128 * 128, &maps.q, full(slot), p * 64,
                     s.h * a.group + w.g0, w.tok0, many);
        }
        if (++slot == NS) {
          slot = 0;
          ++round;
        }
      }
      x = s.first + t1;
    }
    // no copy may be in flight when the CTA's shared memory goes away (other roles may give up after this one's end)
    for (int q = 0; q < NS; ++q)
      if (q < slot || round > 0) bar_drain(full(q), (q < slot ? round : round - 1) & 1);
    for (int q = 0; q < 2; ++q)
      if (q < ks || k_round > 0) bar_drain(k_full(q), (q < ks ? k_round : k_round - 1) & 1);
  } else if (wid == 18) {  // ---------------------------------------------------------------- log-sum-exps
    int slot = 0;
    uint32_t round = 0;
    bool ok = true;
    while (x < x_end && ok) {
      const WtSeg s = wt_find(a, plan, x);
      const int t1 = min(s.first + s.tiles, x_end) - s.first;
      for (int t = x - s.first; t < t1; ++t) {
        const WtTile w = wt_tile(a, plan, s.t_first + t);
        float v[kWtCols / 32];  // on their way while the slot is still in use
#pragma unroll
        for (int q = 0; q < kWtCols / 32; ++q) {
          const int c = lane + 32 * q, i = c / w.gw;
          v[q] = c < w.cols ? a.lse[int64_t(w.tok0 + i) * a.hq + s.h * a.group + w.g0 + (c - i * w.gw)] : INFINITY;
        }
        if (!(ok = bar_wait(l_empty(slot), (round & 1) ^ 1, &waits))) break;
#pragma unroll
        for (int q = 0; q < kWtCols / 32; ++q) minus_lse[slot][lane + 32 * q] = v[q] * -1.4426950408889634f;
        __syncwarp();
        if (lane == 0) bar_arrive(l_full(slot));
        if (++slot == NL) {
          slot = 0;
          ++round;
        }
      }
      x = s.first + t1;
    }
  } else if (wid == 17) {  // ---------------------------------------------------------------- products
    int slot = 0, ks = 0, buf = 0;
    uint32_t round = 0, k_round = 0, b_round = 0;
    bool ok = true;
    while (x < x_end && ok) {
      const WtSeg s = wt_find(a, plan, x);
      const int t1 = min(s.first + s.tiles, x_end) - s.first;
      ok = bar_wait(k_full(ks), k_round & 1, &waits);
      for (int t = x - s.first; t < t1 && ok; ++t) {
        const WtTile w = wt_tile(a, plan, s.t_first + t);
        const uint32_t idesc = mma_idesc((w.cols + 15) / 16 * 16, false);
        ok = bar_wait(full(slot), round & 1, &waits);
        for (int st = 0; st < 2 && ok; ++st) {
          if (!(ok = bar_wait(s_free(st, buf), (b_round & 1) ^ 1, &waits))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t k = desc_low(k_sm + (2 * ks + st) * Sh::kHalf, 16), q = desc_low(ring + slot * Sh::kHalf, 16);
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
              const uint32_t off = (e / 4) * (128 * 128) + (e % 4) * 32;
              mma_ss(tm + st * 256 + buf * 128, k + (off >> 4), q + (off >> 4), idesc, e > 0);
            }
            mma_commit(s_full(st, buf));
            if (st == 1) {
              mma_commit(empty(slot));
              if (t + 1 == t1) mma_commit(k_empty(ks));
            }
          }
          __syncwarp();
        }
        if (++slot == NS) {
          slot = 0;
          ++round;
        }
        if (++buf == 2) {
          buf = 0;
          ++b_round;
        }
      }
      if (++ks == 2) {
        ks = 0;
        ++k_round;
      }
      x = s.first + t1;
    }
    // nothing of the tensor pipe may be in flight when tensor memory is given back
    if (lane == 0) mma_commit(done);
    __syncwarp();
    bar_drain(done, 0);
  } else {  // ---------------------------------------------------------------- the streams' keys
    const int st = (wid >> 2) & 1, mine = wid >> 3, key = tid & 127;
    const uint32_t lane_base = uint32_t((wid & 3) * 32) << 16;
    const float c2 = a.scale * 1.4426950408889634f;
    const uint64_t cc = pair(c2, c2);
    int slot = 0, buf = 0, seg_no = 0;
    uint32_t round = 0, b_round = 0;
    bool ok = true;
    while (x < x_end && ok) {
      const WtSeg s = wt_find(a, plan, x);
      const int t1 = min(s.first + s.tiles, x_end) - s.first;
      const int64_t k = int64_t(s.seg) * kWtKeys + st * 128 + key;
      const int64_t tok_min = a.causal ? k - (a.n - a.m) : 0;  // first token that sees this key
      const float before = mine == 0 && a.acc_in && k < a.n ? a.acc_in[s.h * a.ld_acc_in + k] : 0.f;
      uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
      for (int t = x - s.first; t < t1; ++t) {
        const WtTile w = wt_tile(a, plan, s.t_first + t);
        if (!(ok = bar_wait(l_full(slot), round & 1, &waits))) break;
        if (!(ok = bar_wait(s_full(st, buf), b_round & 1, &waits))) break;
        tc_fence_after();
        const int64_t hid = (tok_min - w.tok0) * w.gw;  // columns before this one do not see the key
        const int c_min = hid < 0 ? 0 : (hid > kWtCols ? kWtCols : int(hid));
        const bool mask = __any_sync(0xffffffffu, c_min > 0) || w.cols < kWtCols;
        const uint32_t ts = tm + lane_base + st * 256 + buf * 128;
#pragma unroll 1
        for (int j = 64 * mine; j < min(64 * mine + 64, w.cols); j += 32) {
          float v[32];
          tmem_ld32(ts + j, v);
          tmem_wait32(v);
          if (mask) {  // also the columns that no product wrote
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (j + q < c_min || j + q >= w.cols) v[q] = -INFINITY;
          }
          const ulonglong2* l = reinterpret_cast<const ulonglong2*>(&minus_lse[slot][j]);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const ulonglong2 l4 = l[q];
            sum[0] = add2(sum[0], ex2_pair(fma2(pair(v[4 * q], v[4 * q + 1]), cc, l4.x)));
            sum[1] = add2(sum[1], ex2_pair(fma2(pair(v[4 * q + 2], v[4 * q + 3]), cc, l4.y)));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(s_free(st, buf));
          bar_arrive(l_empty(slot));
        }
        if (++slot == NL) {
          slot = 0;
          ++round;
        }
        if (++buf == 2) {
          buf = 0;
          ++b_round;
        }
      }
      if (!ok) break;
      float s0, s1;
      unpair(add2(sum[0], sum[1]), &s0, &s1);
      float total = s0 + s1;
      const int par = seg_no & 1;
      const uint32_t use = uint32_t(seg_no >> 1) & 1;  // the parity's pair of barriers serves every other segment
      ++seg_no;
      if (mine == 1) {
        if (!(ok = bar_wait(x_free(par, st), use ^ 1, &waits))) break;
        other[par][st][key] = total;
        __syncwarp();
        if (lane == 0) bar_arrive(x_full(par, st));
      } else {
        if (!(ok = bar_wait(x_full(par, st), use, &waits))) break;
        total += other[par][st][key];
        __syncwarp();
        if (lane == 0) bar_arrive(x_free(par, st));
        if (x == s.first && t1 == s.tiles) {
          if (k < a.n) a.acc_out[s.h * a.ld_acc_out + k] = before + total;
        } else {
          a.sums[(int64_t(blockIdx.x) * 2 + (x_begin < s.first ? 1 : 0)) * kWtKeys + st * 128 + key] = total;
        }
      }
      x = s.first + t1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (waits.gave_up && tid == 0) raise_status(a.status, ZHA_ERR_TIMEOUT);
  if (wid == 17) tmem_free(tm, 512);
}

// Segments cut by CTA borders: block c joins the one that begins in CTA c and ends in a later one.
__global__ void __launch_bounds__(kWtKeys) weights_tc_join_kernel(WeightsArgs a) {
  pdl_wait();
  const int nc = gridDim.x, c = blockIdx.x;
  const WtPlan plan = wt_plan(a, nc);
  const int x0 = plan.sh.begin(c), x1 = plan.sh.begin(c + 1);
  if (x0 >= x1) return;
  const WtSeg s = wt_find(a, plan, x1 - 1);
  if (s.first < x0 || s.first + s.tiles <= x1) return;
  const int64_t k = int64_t(s.seg) * kWtKeys + threadIdx.x;
  if (k >= a.n) return;
  const int last = plan.sh.owner(s.first + s.tiles - 1);
  float sum = 0.f;
  for (int q = c; q <= last; ++q)  // it holds every later share's begin
    sum += a.sums[(int64_t(q) * 2 + (q == c && x0 < s.first ? 1 : 0)) * kWtKeys + threadIdx.x];
  a.acc_out[s.h * a.ld_acc_out + k] = (a.acc_in ? a.acc_in[s.h * a.ld_acc_in + k] : 0.f) + sum;
}

// ------------------------------------------------------------------ host side
namespace {

template <int D> cudaError_t run_weights_tc(const WeightsArgs& a, const WtMaps& maps, int nc, cudaStream_t st) {
  cudaError_t e = allow_smem(weights_tc_kernel<D>, WtShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_after(weights_tc_kernel<D>, dim3(nc), kWtThreads, WtShape<D>::kSmem, st, a, maps);
  if (e != cudaSuccess) return e;
  return launch_after(weights_tc_join_kernel, dim3(nc), kWtKeys, 0, st, a);
}

}  // namespace

uint64_t weights_tc_floats() { return kWtFloats; }

cudaError_t launch_weights_tc(const WeightsArgs& a, int d, cudaStream_t st) {
  WtMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  cudaError_t e = make_rows_map(&maps.k, a.K, d, a.n, a.ld, a.hkv, 128, 1);
  // row tiles: `group` heads of 128 / group tokens, or 128 heads of one token
  if (e == cudaSuccess)
    e = make_rows_map(&maps.q, a.Q, d, a.hq, a.hq, a.m, a.group <= kWtCols ? a.group : kWtCols,
                      a.group <= kWtCols ? kWtCols / a.group : 1);
  if (e != cudaSuccess) return e;
  const int64_t segs = (a.n + kWtKeys - 1) / kWtKeys * a.hkv;
  const int64_t tiles = a.group <= kWtCols ? (a.m + kWtCols / a.group - 1) / (kWtCols / a.group)
                                           : int64_t(a.m) * ((a.group + kWtCols - 1) / kWtCols);
  const int nc = int(min64(148, segs * tiles));
  count_launches(2);
  return d == 128 ? run_weights_tc<128>(a, maps, nc, st) : run_weights_tc<64>(a, maps, nc, st);
}

}  // namespace zha
