// Many query rows over one KV cache on the tensor cores (bf16 configurations): the
// kernel behind zha_prefix_decode and zha_dense_weights.  Work split and partials: zha_rows.cuh.
//
// One CTA per SM, two streams.  A stream is 128 query rows with a 128-row
// accumulator in tensor memory; per tile of 128 keys
//   S = Q K^T           (both from shared memory, 128 x 128 fp32 in tensor memory),
//   P = 2^(S c - m)     (one thread per row: tensor memory -> registers, the row's maximum and sum, and
//                        back over S as bf16),
//   O += P V            (P from tensor memory, V from shared memory).
// P enters the second product as two bf16 parts, hi + lo (S's 128 fp32 columns hold exactly the two), because the
// output is fp32: one part alone leaves 2^-9 of every weight, the two 2^-17.  That makes three products per tile
// instead of two: 3 * 512 cycles at 128 x 128 x 128 against 1024 cycles of exponentials (16 per cycle and SM), so
// with both streams in flight - one in its exponentials while the other's products run - the tensor pipe is the
// limit for many rows, HBM for few.  Measured: 64 sequences behind 256K tokens (4 KV heads of 8, d = 128) 415 us in
// short runs, 1.0e15 tensor operations a second with the third product counted, 475 to 490 us in long ones at the power
// limit; 5,250 cycles per tile of both streams of the 3,072 that its products take.  One sequence (8 rows a head)
// 105 us for 537 MB of K and V, 5.1 TB/s. A segment of more than 128 rows gives each stream its own rows and both
// the same tiles (each K and V tile is loaded once for 256 rows); a smaller one gives both streams the same rows and
// every other tile, and stream 0 joins the two results.
//
// The maximum is lazy: O is rescaled only when a row's maximum has grown by more than 2^20, so weights stay below
// 2^20 (the sums are floating point: nothing is lost) and the usual tile rescales nothing.
//
// The tensor pipe's fp32 accumulation cuts off instead of rounding, so the error of O grows with the number of
// products added to it, 2.1e-8 of O each (measured: 3.7e-5 after 1,760, one stream's share of 256K tokens behind 64
// sequences).  After kFlushTiles tiles (16 products each) O is therefore added to a place of the stream's own in
// global memory (L2) with rounded additions and starts again (5.4e-6 on the same case).  A warpgroup of its own does
// that under the next tile's exponentials, through shared memory by bulk reductions, the streams half a period
// apart.
//
// Roles: warps 0-3 and 4-7 the two streams' rows, warp 8 the TMA loads into a ring of K / V tiles, warps 9 and 10
// issue the two streams' products (a product's operands are five registers that one thread has to provide: one warp
// for both streams took 100 cycles a product, above the 64 it runs). Order of the products per stream: P V of the
// previous tile, then S of the next; a commit after S therefore also says that the earlier P V is complete.
//
// The code of a role runs a few times per launch when lengths are short, and its first run waits for its
// instructions: loops over a row's 128 logits go in two rounds of 2 x 32 columns rather than unrolled.
#include <climits>
#include <cstring>

#include "zha_rows.cuh"
#include "zha_tc.cuh"

namespace zha {

constexpr int kTcKeys = 128;               // keys per tile
constexpr int kTcThreads = 512;
constexpr int kRowRegs = 168, kFewRegs = 88;  // registers a thread: 256 * 168 + 256 * 88 = 512 * 128, the launch's own
constexpr int kTcRows = 256;               // rows of a row block: two streams of 128
constexpr int kFlushTiles = 16;              // tiles of a stream that O adds up
constexpr int kTurnTiles = 4;              // segments of more tiles: the streams take turns
constexpr float kLazyMax = 20.f;           // growth of the maximum (log2) that rescales O

template <int D> struct TcShape {
  static constexpr int kTile = kTcKeys * D * 2;            // bytes of a K or V tile
  static constexpr int kQ = 128 * D * 2;                   // bytes of a stream's Q tile
  static constexpr int kSlots = D == 128 ? 4 : 10;         // ring slots (d = 128: five were no faster)
  static constexpr int kStage = 128 * 64 * 4;              // 64 columns of O on their way to global memory
  static constexpr int kSmem = 2 * kQ + kSlots * kTile + kStage + 1024;  // + alignment
};

struct TcMaps {
  CUtensorMap k, v, ko, vo;
};

// 32 logits of a row from column c0 on, of which the row sees the tile's first `left`.
__device__ __forceinline__ void hide32(float* v, int c0, int left) {
#pragma unroll
  for (int q = 0; q < 32; ++q)
    if (c0 + q >= left) v[q] = -INFINITY;
}
__device__ __forceinline__ float largest32(const float* v) {
  float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int q = 4; q < 28; q += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = max3(m[e], v[q + e], v[q + 4 + e]);
#pragma unroll
  for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], v[28 + e]);
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}
// Kept logits: lg is the row's run of the tile that begins at key k0.  Columns past the last key of a 16-byte piece
// lie in the row's padding.
__device__ __forceinline__ void keep_logits(const RowsArgs& a, float* lg, const float* v, int k0, int c0, float c2) {
#pragma unroll
  for (int q = 0; q < 32; q += 4)
    if (k0 + c0 + q < a.n)
      __stcg(reinterpret_cast<float4*>(lg + c0 + q), make_float4(v[q] * c2, v[q + 1] * c2, v[q + 2] * c2, v[q + 3] * c2));
}

__device__ __forceinline__ void st_shared4(uint32_t at, const float* v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
__device__ __forceinline__ void ld_shared4(uint32_t at, float* v) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(at)
               : "memory");
}
template <typename F> __device__ __forceinline__ void add_row32(float* v, F at) {
#pragma unroll
  for (int q = 0; q < 32; q += 4) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(at(q)));
    v[q] += t.x;
    v[q + 1] += t.y;
    v[q + 2] += t.z;
    v[q + 3] += t.w;
  }
}
// Where the 32 rows from wrow on of stream st add up what they have so far.
__device__ __forceinline__ float* sofar_base(const RowsArgs& a, int st, int wrow, int d) {
  return a.part_tmp + (int64_t(blockIdx.x) * a.rt + st * (a.rt / 2) + wrow) * d;
}

// One share of a segment as every role sees it.
struct TcWork {
  RowsSeg s;
  int t0, cnt;    // its first tile within the segment, its tiles
  int seg_rows;   // rows of the segment's head (prefix) or sequence (own)
  bool both;      // each stream has rows of its own
};

// The next share at or after place *x of the CTA's places, by one full warp; false at their end.
__device__ __forceinline__ bool next_work(const RowsArgs& a, const RowsTotals& tot, int* x, int x_end, TcWork* w) {
  while (*x < x_end) {
    w->s = rows_find(a, tot, *x);
    w->t0 = *x - w->s.first;
    w->cnt = min(w->s.first + w->s.tiles, x_end) - *x;
    *x = w->s.next;
    if (w->cnt > 0) {
      w->seg_rows = w->s.own ? a.m * a.group : a.rows;
      w->both = w->seg_rows - w->s.p * kTcRows > 128;
      return true;
    }
  }
  return false;
}

template <int D, bool PV, bool LG>
__global__ void __launch_bounds__(kTcThreads, 1) rows_tc_kernel(RowsArgs a, const __grid_constant__ TcMaps maps) {
  using Sh = TcShape<D>;
  constexpr int NS = Sh::kSlots, PANELS = D / 64, PANEL = kTcKeys * 128;  // bytes of a 64-wide panel of a tile
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * NS + 25];
  __shared__ float2 x_ml[128];  // stream 1's sums for the join
  __shared__ uint32_t tmem_base;
  __shared__ Waits waits;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t ring = base + 2 * Sh::kQ;
  const uint32_t b0 = smem_u32(bars);
  auto full = [&](int s) { return b0 + 8 * s; };
  auto empty = [&](int s) { return b0 + 8 * (NS + s); };
  // logits ready; without outputs a stream has two buffers for them, the second in place of O
  auto s_full = [&](int s, int buf = 0) { return b0 + 8 * (2 * NS + (buf ? 17 : 0) + s); };
  auto o_full = [&](int s) { return b0 + 8 * (2 * NS + 2 + s); };
  auto q_full = [&](int s) { return b0 + 8 * (2 * NS + 4 + s); };
  auto p_full = [&](int s, int half) { return b0 + 8 * (2 * NS + 6 + 2 * s + half); };
  const uint32_t fix = b0 + 8 * (2 * NS + 10), done = fix + 8, x_full = fix + 16, x_free = fix + 24, x_may = fix + 32;
  auto o_chunk = [&](int s) { return b0 + 8 * (2 * NS + 19 + s); };     // O is complete up to a point where it starts again
  auto o_free = [&](int s) { return b0 + 8 * (2 * NS + 21 + s); };      // and has been read
  auto flush_done = [&](int s) { return b0 + 8 * (2 * NS + 23 + s); };  // and added to global memory
  auto turn = [&](int s) { return fix + 40 + 8 * s; };  // the other stream has weighed its tile
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

  if (wid == 11) {
    if (lane == 0) {
      for (int s = 0; s < NS; ++s) {
        bar_init(full(s), 1);
        bar_init(empty(s), 2);  // both streams
      }
      for (int s = 0; s < 2; ++s) {
        bar_init(s_full(s), 1);
        bar_init(s_full(s, 1), 1);
        bar_init(o_full(s), 1);
        bar_init(q_full(s), 4);
        bar_init(o_chunk(s), 1);
        bar_init(o_free(s), 4);
        bar_init(flush_done(s), 4);
        bar_init(p_full(s, 0), 4);
        bar_init(p_full(s, 1), 4);
      }
      bar_init(fix, 1);
      bar_init(done, 2);
      bar_init(x_full, 4);
      bar_init(x_free, 4);
      bar_init(x_may, 4);
      bar_init(turn(0), 4);
      bar_init(turn(1), 4);
      waits.gave_up = 0;
      waits.limit = a.wait_limit;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    tmem_alloc(smem_u32(&tmem_base), 512);
  }
  pdl_trigger();
  pdl_wait();  // everything above runs under the end of the kernel before
  const RowsTotals tot = rows_totals(a);
  const int x_begin = tot.sh.begin(blockIdx.x), x_end = tot.sh.begin(blockIdx.x + 1);
  int x = x_begin;
  TcWork w;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;

  if (wid >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (wid == 8) {  // ---------------------------------------------------------------- loads
      int slot = 0;
      uint32_t round = 0, fix_phase = 0;
      bool ok = true;
      const uint64_t once = l2_evict_first(), many = l2_evict_normal();
      int pend_slot = -1, pend_row = 0;  // a V tile whose rows from pend_row on are still to be cleared
      auto clear_pending = [&]() {
        if (pend_slot < 0) return true;
        if (!bar_wait(fix, fix_phase, &waits)) return false;
        fix_phase ^= 1;
        const uint32_t dst = ring + pend_slot * Sh::kTile + pend_row * 128;
        const int per = (kTcKeys - pend_row) * 8;
#pragma unroll 1
        for (int p = 0; p < PANELS; ++p)
#pragma unroll 1
          for (int q = lane; q < per; q += 32)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + p * PANEL + q * 16), "r"(0) : "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(full(pend_slot));
        pend_slot = -1;
        return true;
      };
      while (ok && next_work(a, tot, &x, x_end, &w)) {
        const int lag = w.both ? 1 : 2;
        // tiles that no other row block reads go first when L2 needs room (kept logits stay)
        const uint64_t policy = w.s.own || a.pp == 1 ? once : many;
        const CUtensorMap* mk = w.s.own ? &maps.ko : &maps.k;
        const CUtensorMap* mv = w.s.own ? &maps.vo : &maps.v;
        const int plane = w.s.own ? w.s.b * a.hkv + w.s.h : w.s.h;
        const int len = int(w.s.own ? own_tokens(a, w.s.b) : a.n);
#pragma unroll 1
        for (int i = 0; i < 2 * (w.cnt + lag) && ok; ++i) {
          const bool kv = !(i & 1);  // V of tile i/2 - lag, then K of tile i/2: the order of their use
          const int t = (i >> 1) - (kv ? lag : 0);
          if (kv ? (!PV || t < 0) : t >= w.cnt) continue;
          const int k0 = (w.t0 + t) * kTcKeys;
          // rows of V past a sequence's end hold anything (0 * NaN is NaN): cleared before the product sees them,
          // once the copy has landed; meanwhile the next copies start, as long as none has to wait.  Past the
          // prefix's end the tensor map ends, so the copy itself fills zeros.
          const bool clear = kv && w.s.own && k0 + kTcKeys > len;
          if ((clear || !bar_look(empty(slot), (round & 1) ^ 1)) && !(ok = clear_pending())) break;
          if (!(ok = bar_wait(empty(slot), (round & 1) ^ 1, &waits))) break;
          const uint32_t dst = ring + slot * Sh::kTile;
          const uint32_t bar = clear ? fix : full(slot);
          if (lane == 0) {
            bar_expect(bar, Sh::kTile);
#pragma unroll
            for (int p = 0; p < PANELS; ++p) tma_load(dst + p * PANEL, kv ? mv : mk, bar, p * 64, k0, plane, policy);
          }
          if (clear) {
            pend_slot = slot;
            pend_row = len - k0;
          }
          if (++slot == NS) {
            slot = 0;
            ++round;
          }
        }
      }
      if (ok) clear_pending();
      // no copy may be in flight when the CTA's shared memory goes away (other roles may give up after this one's end)
      for (int q = 0; q < NS; ++q) {
        const uint32_t r = q < slot ? round : round - 1;  // the slot's last use
        if (q < slot || round > 0) bar_drain(q == pend_slot ? fix : full(q), q == pend_slot ? fix_phase : r & 1);
      }
    } else if (wid == 9 || wid == 10) {  // ---------------------------------------------------------------- products
      const int st = wid - 9;
      constexpr uint32_t id_s = mma_idesc(kTcKeys, false), id_o = mma_idesc(D, true);
      const uint32_t ts = tm + st * 128, to = tm + 256 + st * D;
      const uint32_t q_lo = desc_low(base + st * Sh::kQ, 16);
      const uint32_t k_lo = desc_low(ring, 16), v_lo = desc_low(ring, PANEL);
      int slot = 0;
      uint32_t round = 0, p_phase = 0, q_phase = 0, b_round = 0, o_phase = 0;
      int buf = 0;
      bool ok = true;
      while (ok && next_work(a, tot, &x, x_end, &w)) {
        const int lag = w.both ? 1 : 2;
        if (!(ok = bar_wait(q_full(st), q_phase, &waits))) break;
        q_phase ^= 1;
        if (!w.both && w.cnt == 1 && st == 1 && lane == 0) bar_arrive(o_full(1));  // no tile for stream 1: nothing to wait for
        int room = kFlushTiles - st * (kFlushTiles / 2);  // tiles until O starts again
        bool fresh = true, first = true;
#pragma unroll 1
        for (int i = 0; i < w.cnt + lag && ok; ++i) {
          const bool mine = w.both || (i & 1) == st;
          if (i >= lag && PV) {
            if (!(ok = bar_wait(full(slot), round & 1, &waits))) break;
            if (mine) {
              if (fresh && !first && !(ok = bar_wait(o_free(st), o_phase, &waits))) break;
              if (fresh && !first) o_phase ^= 1;
              first = false;
              // the weights come in two halves of 64 keys: the products of the first run under the exponentials of
              // the second
              const uint32_t v = v_lo + slot * (Sh::kTile >> 4);
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                if (!(ok = bar_wait(p_full(st, half), p_phase, &waits))) break;
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                  for (int k = half * 4; k < half * 4 + 4; ++k)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                      mma_ts(to, ts + (k / 2) * 32 + part * 16 + (k & 1) * 8, v + k * (2048 >> 4), id_o,
                             k || part ? 1u : uint32_t(!fresh));
                }
                __syncwarp();
              }
              if (!ok) break;
              p_phase ^= 1;
              fresh = --room == 0;
              if (fresh) room = kFlushTiles;
              if (lane == 0) {
                if (fresh && i + (w.both ? 1 : 2) < w.cnt + lag) mma_commit(o_chunk(st));
                mma_commit(empty(slot));
                if (i + lag >= w.cnt + lag) mma_commit(o_full(st));
              }
            } else if (lane == 0) {
              bar_arrive(empty(slot));
            }
            __syncwarp();
            if (++slot == NS) {
              slot = 0;
              ++round;
            }
          }
          if (i < w.cnt) {
            if (!(ok = bar_wait(full(slot), round & 1, &waits))) break;
            if (mine) {
              if (!PV && !(ok = bar_wait(p_full(st, buf), (b_round & 1) ^ 1, &waits))) break;  // the buffer has been read
              tc_fence_after();
              if (lane == 0) {
                const uint32_t k = k_lo + slot * (Sh::kTile >> 4);
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                  const uint32_t off = ((e / 4) * PANEL + (e % 4) * 32) >> 4;
                  mma_ss(ts + (PV ? 0 : buf * 256), q_lo + off, k + off, id_s, e ? 1u : 0u);
                }
                mma_commit(s_full(st, PV ? 0 : buf));
                mma_commit(empty(slot));
              }
              if (!PV && ++buf == 2) {
                buf = 0;
                ++b_round;
              }
            } else if (lane == 0) {
              bar_arrive(empty(slot));
            }
            __syncwarp();
            if (++slot == NS) {
              slot = 0;
              ++round;
            }
          }
        }
      }
      // nothing of the tensor pipe may be in flight when tensor memory is given back
      if (lane == 0) mma_commit(done);
      __syncwarp();
      bar_drain(done, 0);
    } else if (wid == 11) {
      if (blockIdx.x == 0) rows_publish(a, tot);
    } else if (PV) {  // ---------------------------------------------------------------- O to global memory
      const int wrow = (wid & 3) * 32;
      const uint32_t stage = ring + NS * Sh::kTile + wrow * 256;
      uint32_t phase[2] = {0, 0};
      bool ok = true;
      while (ok && next_work(a, tot, &x, x_end, &w)) {
        // the streams' flushes in the order of their tiles: stream 1 after kFlushTiles / 2, stream 0 after
        // kFlushTiles, ...
        const int n0 = w.both ? w.cnt : (w.cnt + 1) / 2, n1 = w.both ? w.cnt : w.cnt / 2;
#pragma unroll 1
        for (int f = 0; f * (kFlushTiles / 2) + kFlushTiles / 2 < max(n0, n1) && ok; ++f) {
          const int st = (f & 1) ^ 1;
          if ((f + 1) * (kFlushTiles / 2) >= (st ? n1 : n0)) continue;  // the stream ends before
          if (!(ok = bar_wait(o_chunk(st), phase[st], &waits))) break;
          phase[st] ^= 1;
          tc_fence_after();
          const int nrows = min(128, w.seg_rows - w.s.p * kTcRows - (w.both ? st * 128 : 0));
          const uint32_t to = tm + (uint32_t(wrow) << 16) + 256 + st * D;
          float* dst = sofar_base(a, st, wrow, D);
          if (wrow < nrows) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 64) {
#pragma unroll 1
              for (int j = 0; j < 64; j += 32) {
                float v[32];
                tmem_ld32(to + c0 + j, v);
                tmem_wait32(v);
#pragma unroll
                for (int q = 0; q < 8; ++q) st_shared4(stage + lane * 256 + ((((j >> 2) + q) ^ (lane & 7)) << 4), v + 4 * q);
              }
              if (c0 + 64 == D) {  // all of O has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(o_free(st));
              }
              fence_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (f < 2) bulk_store(dst + c0 * 32, stage, 32 * 256);
                else bulk_add(dst + c0 * 32, stage, 32 * 256);
                bulk_commit();
                if (c0 + 64 == D) bulk_wait_all();  // before the next addition to the same place, and before anyone reads it
                else bulk_wait_read();
              }
              __syncwarp();
            }
            asm volatile("fence.proxy.async;" ::: "memory");
          } else if (lane == 0) {
            bar_arrive(o_free(st));
          }
          if (lane == 0) bar_arrive(flush_done(st));
        }
      }
    }
  } else {  // ---------------------------------------------------------------- the streams' rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    const int st = wid >> 2, row = tid & 127, wrow = (wid & 3) * 32;
    const uint32_t lane_base = uint32_t(wrow) << 16;
    const uint32_t ts = tm + lane_base + st * 128, to = tm + lane_base + 256 + st * D;
    const float c2 = a.scale * 1.4426950408889634f;  // weights as powers of two
    const uint64_t cc = pair(c2, c2), minus = pair(-1.f, -1.f);
    uint32_t s_phase = 0, o_phase = 0, x_phase = 0, t_phase = 0, f_phase = 0;
    int buf = 0;
    bool ok = true;
    while (ok && next_work(a, tot, &x, x_end, &w)) {
      const int r0 = w.s.p * kTcRows + (w.both ? st * 128 : 0);  // the stream's first row
      const int nrows = min(128, w.seg_rows - r0);
      const int row_off = w.s.own ? w.s.b * a.m * a.group : 0;
      // queries to shared memory, every warp its own rows: they are where its results leave from, and no other warp
      // waits for that
      auto load_queries = [&]() {
        constexpr int CH = D / 8, RP = 32 / CH;  // 16-byte pieces of a row, rows per pass of a warp
        const int c = lane % CH, rq = wrow + lane / CH;
        const __nv_bfloat16* Qp = static_cast<const __nv_bfloat16*>(a.Q) + c * 8;
        const uint32_t dst = base + st * Sh::kQ + (c / 8) * (128 * 128);
#pragma unroll 1
        for (int g = 0; g < CH; g += 8) {  // eight loads in flight
          uint4 v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int r = (g + q) * RP + rq;
            v[q] = r < nrows ? *reinterpret_cast<const uint4*>(Qp + row_index(a, w.s.h, row_off + r0 + r) * D)
                             : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int r = (g + q) * RP + rq;
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                         "r"(v[q].x), "r"(v[q].y), "r"(v[q].z), "r"(v[q].w)
                         : "memory");
          }
        }
      };
      load_queries();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(q_full(st));
      // (padding rows: no limit, so that they never ask for the masked path)
      const int lim = row >= nrows ? INT_MAX : int(w.s.own ? own_limit(a, own_tokens(a, w.s.b), r0 + row) : prefix_limit(a, r0 + row));
      const bool active = wrow < nrows;  // a warp of padding rows leaves its weights alone: they reach no valid row
      float m_ref = -INFINITY, l_run = 0.f;
      bool flushed = false, pending = false;  // O has been added to global memory; maybe not done yet
      // where the rows' results go: a partial, or the result itself where this CTA's share holds all tiles
      const bool whole = !a.has_own && w.t0 == 0 && w.cnt == w.s.tiles;
      const int64_t pr = part_row(a, blockIdx.x, w.s.own, w.s.id, x_begin < w.s.first) + (w.both ? st * 128 : 0) + row;
      const int64_t ri = row < nrows ? row_index(a, w.s.h, row_off + r0 + row) : 0;
      // and where O is added up meanwhile, in the order it leaves shared memory: 64 columns, rows, swizzled 16-byte
      // pieces
      float* const sofar = sofar_base(a, st, wrow, D);
      auto sofar_at = [&](int col) {
        return sofar + (col >> 6) * (32 * 64) + lane * 64 + ((((col & 63) >> 2) ^ (lane & 7)) << 2);
      };
      constexpr int HC = D / 2, LN = HC / 4;  // columns of half a row, lanes for one
      // 16-byte piece k of the half row from column c0 on, of row r: over both streams' queries, or over the
      // stream's own
      auto cell = [&](bool all, int c0, int k, int r) {
        return all ? base + r * (D * 4) + c0 * 4 + ((k ^ (r & 7)) << 4)
                   : base + st * Sh::kQ + (k >> 3) * (128 * 128) + r * 128 + (((k & 7) ^ (r & 7)) << 4);
      };
      const int step = w.both ? 1 : 2, i0 = w.both ? 0 : st;
      if constexpr (PV) {
        // Streams take turns: a tile may begin once the other stream has handed over half of its own.  Left alone
        // they fall into step, and the tensor pipe idles while both weigh (256K tokens behind 64 sequences: 413 us,
        // whole turns 400, half turns 380).
        const bool turns = w.cnt > kTurnTiles;
        int room = kFlushTiles - st * (kFlushTiles / 2);  // tiles until O starts again
        bool fresh = true, first_tile = true;
#pragma unroll 1
        for (int i = i0; i < w.cnt; i += step) {
          if (turns && (st || i != i0)) {
            if (!(ok = bar_wait(turn(st), t_phase, &waits))) break;
            t_phase ^= 1;
          }
          if (!(ok = bar_wait(s_full(st), s_phase, &waits))) break;
          s_phase ^= 1;
          tc_fence_after();
          if (fresh && !first_tile) pending = flushed = true;  // O is being added to global memory
          // before this tile's weights can complete O and have it added again, every warp has seen the time before
          if (pending && room == 1) {
            if (!(ok = bar_wait(flush_done(st), f_phase, &waits))) break;
            f_phase ^= 1;
            pending = false;
          }
          if (active) {
            const int left = lim - (w.t0 + i) * kTcKeys;  // keys of the tile that the row sees
            const bool mask = __any_sync(0xffffffffu, left < kTcKeys);
            float va[32], vb[32];
            float mx;
            {
              float vc[32], vd[32];
              tmem_ld32(ts, va);
              tmem_ld32(ts + 32, vb);
              tmem_ld32(ts + 64, vc);
              tmem_ld32(ts + 96, vd);
              tmem_wait32(va);
              tmem_wait32(vb);
              tmem_wait32(vc);
              tmem_wait32(vd);
              if (mask) {
                hide32(va, 0, left);
                hide32(vb, 32, left);
                hide32(vc, 64, left);
                hide32(vd, 96, left);
              }
              mx = fmaxf(fmaxf(largest32(va), largest32(vb)), fmaxf(largest32(vc), largest32(vd)));
            }
            tmem_ld32(ts, va);  // again, chunk by chunk, for the exponentials
            const float m_new = mx * c2;
            const bool grow = m_new > m_ref + kLazyMax || (m_ref == -INFINITY && m_new > -INFINITY);
            if (__any_sync(0xffffffffu, grow)) {
              const float up = grow ? m_new : m_ref;
              const float sc = m_ref == -INFINITY ? 0.f : ex2(m_ref - up);
              if (flushed) {  // what has left O already
                if (pending) {
                  if (!(ok = bar_wait(flush_done(st), f_phase, &waits))) {
                    tmem_wait32(va);  // the load above must not outlive the loop
                    break;
                  }
                  f_phase ^= 1;
                  pending = false;
                }
                if (grow) {
#pragma unroll 1
                  for (int j = 0; j < D; j += 32) {  // eight pieces on their way
#pragma unroll
                    for (int q = 0; q < 32; q += 4)
                      *reinterpret_cast<float4*>(vb + q) = __ldcg(reinterpret_cast<const float4*>(sofar_at(j + q)));
#pragma unroll
                    for (int q = 0; q < 32; q += 4) {
#pragma unroll
                      for (int e = 0; e < 4; ++e) vb[q + e] = m_ref == -INFINITY ? 0.f : vb[q + e] * sc;
                      __stcg(reinterpret_cast<float4*>(sofar_at(j + q)), make_float4(vb[q], vb[q + 1], vb[q + 2], vb[q + 3]));
                    }
                  }
                  __threadfence();
                  asm volatile("fence.proxy.async;" ::: "memory");
                }
                __syncwarp();
              }
              if (!fresh) {
#pragma unroll 1
                for (int j = 0; j < D; j += 32) {
                  tmem_ld32(to + j, vb);
                  tmem_wait32(vb);
                  if (grow) {
#pragma unroll
                    for (int q = 0; q < 32; ++q) vb[q] = m_ref == -INFINITY ? 0.f : vb[q] * sc;
                  }
                  tmem_st32(to + j, reinterpret_cast<const uint32_t*>(vb));
                }
              }
              if (grow) {
                l_run *= sc;
                m_ref = up;
              }
            }
            const float mb = m_ref == -INFINITY ? 0.f : m_ref;
            const uint64_t mm = pair(-mb, -mb);
            uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
            // kept logits: the row's own run of the tile (columns past the last key lie in the padding of the row)
            float* lg = LG && row < nrows
                            ? a.logits + (int64_t(w.s.h) * a.rows + r0 + row) * a.ld_logits + int64_t(w.t0 + i) * kTcKeys
                            : nullptr;
            auto weigh = [&](const float* v, int c0) {  // 32 keys: their weights' hi parts, then their lo parts, over the logits
              uint32_t o[32];
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                const uint64_t e = fma2(pair(v[2 * q], v[2 * q + 1]), cc, mm);
                const uint64_t p = ex2_pair(e);
                sum[q & 1] = add2(sum[q & 1], p);
                float p0, p1;
                unpair(p, &p0, &p1);
                o[q] = pack_bf16(p0, p1);
                unpair(fma2(pair(__uint_as_float(o[q] << 16), __uint_as_float(o[q] & 0xffff0000u)), minus, p), &p0, &p1);
                o[16 + q] = pack_bf16(p0, p1);
              }
              tmem_st32(ts + c0, o);
              if (LG && lg) keep_logits(a, lg, v, (w.t0 + i) * kTcKeys, c0, c2);
            };
#pragma unroll 1
            for (int j = 0; j < kTcKeys; j += 64) {
              tmem_wait32(va);
              tmem_ld32(ts + j + 32, vb);
              if (mask) hide32(va, j, left);
              weigh(va, j);
              tmem_wait32(vb);
              if (j == 0) tmem_ld32(ts + 64, va);
              if (mask) hide32(vb, j + 32, left);
              weigh(vb, j + 32);
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                bar_arrive(p_full(st, j >> 6));
                if (turns && j == 0) bar_arrive(turn(st ^ 1));
              }
            }
            float s0, s1;
            unpair(add2(sum[0], sum[1]), &s0, &s1);
            l_run += s0 + s1;
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              bar_arrive(p_full(st, 0));
              bar_arrive(p_full(st, 1));
              if (turns) bar_arrive(turn(st ^ 1));
            }
          }
          first_tile = false;
          fresh = --room == 0;
          if (fresh) room = kFlushTiles;
        }
        // turns of the other stream that this one has no tile to wait for: the last one of stream 1, for stream 0
        // and of stream 0 for a stream 1 with one tile less
        if (ok && turns && (st == 0 ? w.both || !(w.cnt & 1) : !w.both && (w.cnt & 1))) {
          if (!(ok = bar_wait(turn(st), t_phase, &waits))) break;
          t_phase ^= 1;
        }
      } else {
#pragma unroll 1
        for (int i = i0; i < w.cnt; i += step) {  // only the sums
          if (!(ok = bar_wait(s_full(st, buf), s_phase, &waits))) break;
          tc_fence_after();
          if (active) {
            const int left = lim - (w.t0 + i) * kTcKeys;  // keys of the tile that the row sees
            const bool mask = __any_sync(0xffffffffu, left < kTcKeys);
            const uint32_t tb = ts + buf * 256;
            float* lg = LG && row < nrows
                            ? a.logits + (int64_t(w.s.h) * a.rows + r0 + row) * a.ld_logits + int64_t(w.t0 + i) * kTcKeys
                            : nullptr;
            float v[kTcKeys];
#pragma unroll
            for (int j = 0; j < kTcKeys; j += 32) tmem_ld32(tb + j, v + j);
#pragma unroll
            for (int j = 0; j < kTcKeys; j += 32) tmem_wait32(v + j);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_full(st, buf));  // the buffer has been read
            if (mask) {
#pragma unroll
              for (int j = 0; j < kTcKeys; j += 32) hide32(v + j, j, left);
            }
            const float m_new = fmaxf(fmaxf(largest32(v), largest32(v + 32)), fmaxf(largest32(v + 64), largest32(v + 96))) * c2;
            if (m_new > m_ref + kLazyMax || (m_ref == -INFINITY && m_new > -INFINITY)) {
              l_run *= m_ref == -INFINITY ? 0.f : ex2(m_ref - m_new);
              m_ref = m_new;
            }
            const float mb = m_ref == -INFINITY ? 0.f : m_ref;
            const uint64_t mm = pair(-mb, -mb);
            uint64_t sum[4] = {pair(0.f, 0.f), pair(0.f, 0.f), pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
            for (int q = 0; q < kTcKeys / 2; ++q)
              sum[q & 3] = add2(sum[q & 3], ex2_pair(fma2(pair(v[2 * q], v[2 * q + 1]), cc, mm)));
            float s0, s1;
            unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), &s0, &s1);
            l_run += s0 + s1;
            if (LG && lg) {
#pragma unroll
              for (int j = 0; j < kTcKeys; j += 32) keep_logits(a, lg, v + j, (w.t0 + i) * kTcKeys, j, c2);
            }
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_full(st, buf));
          }
          if (++buf == 2) {
            buf = 0;
            s_phase ^= 1;
          }
        }
      }
      if (!ok) break;
      if (PV || i0 >= w.cnt) {  // also without work: the stream stays within one segment of its products' warp
        if (!(ok = bar_wait(o_full(st), o_phase, &waits))) break;
        o_phase ^= 1;
        tc_fence_after();
      }
      // streams that shared the rows: stream 1 leaves its sums and rows where the queries lay, stream 0 joins them
      const bool join = !w.both && w.cnt > 1;
      if (pending) {
        if (!(ok = bar_wait(flush_done(st), f_phase, &waits))) break;
        f_phase ^= 1;
      }
      const bool added = flushed;
      flushed = flushed && row < nrows;
      float other_l = 0.f, mine_s = 1.f, other_s = 0.f;
      if (join) {
        if (st == 1) {
          if (!(ok = bar_wait(x_may, x_phase, &waits))) break;  // stream 0's products still read its queries
          if (active) {
            if (PV) {
#pragma unroll 1
              for (int j = 0; j < D; j += 32) {
                float v[32];
                tmem_ld32(to + j, v);
                tmem_wait32(v);
                if (flushed) add_row32(v, [&](int c) { return sofar_at(j + c); });
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  st_shared4(cell(true, j & ~(HC - 1), ((j & (HC - 1)) >> 2) + q, row), v + 4 * q);
              }
            }
            x_ml[row] = make_float2(m_ref, l_run);
          }
          __syncwarp();
          if (lane == 0) bar_arrive(x_full);
        } else {
          __syncwarp();
          if (lane == 0) bar_arrive(x_may);
          if (!(ok = bar_wait(x_full, x_phase, &waits))) break;
          if (active) {
            const float2 ml = x_ml[row];
            const bool none = ml.x == -INFINITY && ml.y == 0.f;
            const float up = none ? m_ref : fmaxf(m_ref, ml.x);
            mine_s = m_ref == -INFINITY ? (l_run == 0.f ? 0.f : 1.f) : ex2(m_ref - up);
            other_s = none ? 0.f : ex2(ml.x - up);
            other_l = ml.y;
            l_run = l_run * mine_s + (none ? 0.f : other_l * other_s);
            m_ref = up;
          }
        }
      }
      if (active && (w.both || st == 0)) {
        float inv = mine_s;
        if (row < nrows) {
          if (whole) {
            const float n = l_run == 0.f ? 0.f : 1.f / l_run;
            inv *= n;
            other_s *= n;
            if (a.lse) a.lse[ri] = l_run > 0.f ? (m_ref + log2f(l_run)) * 0.6931471805599453f : (l_run == 0.f ? -INFINITY : l_run);
          } else {
            a.part_ml[pr] = make_float2(m_ref, l_run);
          }
        }
        if (PV) {
          // through shared memory, half a row at a time, so that it leaves in whole runs (one thread's row straight
          // from its registers took 4 us a segment): over the other stream's rows when joining, else over the
          // stream's own queries, which no product reads any more
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += HC) {
#pragma unroll 1
            for (int j = 0; j < HC; j += 32) {
              float v[32];
              tmem_ld32(to + c0 + j, v);
              tmem_wait32(v);
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const uint32_t at = cell(join, c0, (j >> 2) + q, row);
                float o[4] = {v[4 * q] * inv, v[4 * q + 1] * inv, v[4 * q + 2] * inv, v[4 * q + 3] * inv};
                if (join && other_s != 0.f) {
                  float t[4];
                  ld_shared4(at, t);
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[e] = fmaf(t[e], other_s, o[e]);
                }
                st_shared4(at, o);
              }
            }
            __syncwarp();
            const int ln = lane % LN;
            constexpr int RS = 32 / LN, BATCH = 8;  // rows at a time, and of these on their way
#pragma unroll 1
            for (int rb = lane / LN; rb - lane / LN < min(32, nrows - wrow); rb += BATCH * RS) {
              float4 t[BATCH];
#pragma unroll
              for (int u = 0; u < BATCH; ++u) {
                const int r = rb + u * RS;
                t[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (added && wrow + r < nrows)  // what left O before
                  t[u] = __ldcg(reinterpret_cast<const float4*>(sofar + (c0 >> 6) * (32 * 64) + r * 64 +
                                                                (((((c0 & 63) >> 2) + ln) ^ (r & 7)) << 2)));
              }
#pragma unroll
              for (int u = 0; u < BATCH; ++u) {
                const int r = rb + u * RS, rr = wrow + r;
                const float f = __shfl_sync(0xffffffffu, inv, r);
                if (rr < nrows) {
                  float o[4];
                  ld_shared4(cell(join, c0, ln, rr), o);
                  float* dst = whole ? a.O + row_index(a, w.s.h, row_off + r0 + rr) * D : a.part + (pr - row + rr) * D;
                  *reinterpret_cast<float4*>(dst + c0 + ln * 4) =
                      make_float4(fmaf(t[u].x, f, o[0]), fmaf(t[u].y, f, o[1]), fmaf(t[u].z, f, o[2]), fmaf(t[u].w, f, o[3]));
                }
              }
            }
            __syncwarp();
          }
        }
      }
      if (join) {  // the next queries go where the rows lie
        if (st == 0) {
          __syncwarp();
          if (lane == 0) bar_arrive(x_free);
        }
        if (!(ok = bar_wait(x_free, x_phase, &waits))) break;
        x_phase ^= 1;
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (waits.gave_up && tid == 0) raise_status(a.status, ZHA_ERR_TIMEOUT);
  if (wid == 11) tmem_free(tm, 512);
}

// ------------------------------------------------------------------ host side
namespace {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

}  // namespace

cudaError_t make_rows_map(CUtensorMap* map, const void* base, int d, int64_t rows, int64_t plane_rows, int64_t planes,
                          int box_rows, int box_planes) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(rows), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(plane_rows) * d * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(box_rows), cuuint32_t(box_planes)}, el[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, el,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

template <int D, bool PV, bool LG> cudaError_t run_tc_as(const RowsArgs& a, const TcMaps& maps, cudaStream_t st) {
  const cudaError_t e = allow_smem(rows_tc_kernel<D, PV, LG>, TcShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_after(rows_tc_kernel<D, PV, LG>, dim3(a.nc), kTcThreads, TcShape<D>::kSmem, st, a, maps);
}

template <int D> cudaError_t run_tc(const RowsArgs& a, const TcMaps& maps, cudaStream_t st) {
  if (a.logits) return a.O ? run_tc_as<D, true, true>(a, maps, st) : run_tc_as<D, false, true>(a, maps, st);
  return a.O ? run_tc_as<D, true, false>(a, maps, st) : run_tc_as<D, false, false>(a, maps, st);
}

}  // namespace

cudaError_t launch_rows_tc(const RowsArgs& a, int d, cudaStream_t st) {
  TcMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  cudaError_t e = cudaSuccess;
  if (a.n > 0) {
    e = make_rows_map(&maps.k, a.K, d, a.n, a.ld, a.hkv, kTcKeys, 1);
    if (e == cudaSuccess && a.V) e = make_rows_map(&maps.v, a.V, d, a.n, a.ld, a.hkv, kTcKeys, 1);
  }
  if (e == cudaSuccess && a.has_own) {
    e = make_rows_map(&maps.ko, a.Ko, d, a.ld_own, a.ld_own, int64_t(a.B) * a.hkv, kTcKeys, 1);
    if (e == cudaSuccess) e = make_rows_map(&maps.vo, a.Vo, d, a.ld_own, a.ld_own, int64_t(a.B) * a.hkv, kTcKeys, 1);
  }
  if (e != cudaSuccess) return e;
  return d == 128 ? run_tc<128>(a, maps, st) : run_tc<64>(a, maps, st);
}

void tc_plan(int64_t rows, int64_t mg, int64_t ld_own, RowsPlan* p) {
  p->rb_log = 8;
  p->kt_log = 7;
  // queries, first loads and the write-out of a segment take about as long as four tiles of one stream's rows each,
  // three of both (32K behind 16 sequences: 2 places 44 us, 4 places 39, 8 places 40; a 4,099-token prompt: 2 places
  // 126, 3 places 120, 4 places 122)
  p->extra = rows > 128 ? 3 : 4;
  p->pp = int((rows + kTcRows - 1) / kTcRows);
  p->po = ld_own > 0 ? int((mg + kTcRows - 1) / kTcRows) : 0;
  p->rp = int(min64(rows, kTcRows));
  p->ro = int(min64(mg, kTcRows));
  p->rt = 2 * int((min64(rows, 128) + 31) / 32 * 32);  // both streams, whole warps
}

}  // namespace zha
