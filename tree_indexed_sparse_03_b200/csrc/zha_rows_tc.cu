// Many query rows over one KV cache on the tensor cores (bf16 configurations): the
// kernel behind zha_prefix_decode and zha_dense_weights.  Work split and partials: zha_rows.cuh.
//
// One CTA per SM, two streams.  A stream is 128 query rows with a 128-row
// accumulator in tensor memory; per tile of 128 keys
//   S = Q K^T           (both from shared memory, 128 x 128 fp32 in tensor memory),
//   P = 2^(S c - m)     (one thread per row: tensor memory -> registers, the row's maximum and sum, and
//                        back over S as bf16),
//   O += P V            (P from tensor memory, V from shared memory).
// P enters the second product as two bf16 parts, hi + lo (S's 128 fp32 columns hold exactly the
// two), because the output is fp32: one part alone leaves 2^-9 of every weight, the two 2^-17.  That
// makes three products per tile instead of two: 3 * 512 cycles at 128 x 128 x 128 against 1024 cycles of exponentials
// (16 per cycle and SM), so with both streams in flight - one in its exponentials while the other's products
// run - the tensor pipe is the limit for many rows, HBM for few.
// A segment of more than 128 rows gives each stream its own rows and both the same tiles (each K and V
// tile is loaded once for 256 rows); a smaller one gives both streams the same rows and every other tile,
// and their two results are joined with the other partials.
//
// The maximum is lazy: O is rescaled in tensor memory only when a row's maximum has grown by more than 2^8, so
// weights stay below 2^8 and the usual tile rescales nothing.
//
// Roles: warps 0-3 and 4-7 the two streams' rows, warp 8 the TMA loads into a ring of K / V
// tiles, warp 9 issues the products.  A row's 128 logits stay in one thread's registers, so the streams' warps take
// registers over from the others.  Order of the products per stream: P V of the previous tile, then
// S of the next; a commit after S therefore also says that the earlier P V is complete.
#include <cstring>

#include "zha_rows.cuh"
#include "zha_tc.cuh"

namespace zha {

constexpr int kTcKeys = 128;               // keys per tile
constexpr int kTcThreads = 384;            // three warpgroups, the third one's last two warps idle
constexpr int kRowRegs = 224, kFewRegs = 56;  // registers a thread: 2 * 128 * 224 + 128 * 56 = 384 * 168, the launch's own
constexpr int kTcRows = 256;               // rows of a row block: two streams of 128
constexpr float kLazyMax = 8.f;            // growth of the maximum (log2) that rescales O

template <int D> struct TcShape {
  static constexpr int kTile = kTcKeys * D * 2;            // bytes of a K or V tile
  static constexpr int kQ = 128 * D * 2;                   // bytes of a stream's Q tile
  static constexpr int kSlots = D == 128 ? 5 : 10;         // ring slots
  static constexpr int kSmem = 2 * kQ + kSlots * kTile + 1024;  // + alignment
};

struct TcMaps {
  CUtensorMap k, v, ko, vo;
};

template <int D, bool PV>
__global__ void __launch_bounds__(kTcThreads, 1) rows_tc_kernel(RowsArgs a, const __grid_constant__ TcMaps maps) {
  using Sh = TcShape<D>;
  constexpr int NS = Sh::kSlots, PANELS = D / 64;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * NS + 12];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int gave_up;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t q_sm[2] = {base, base + Sh::kQ};
  const uint32_t ring = base + 2 * Sh::kQ;
  const uint32_t b0 = smem_u32(bars);
  auto full = [&](int s) { return b0 + 8 * s; };
  auto empty = [&](int s) { return b0 + 8 * (NS + s); };
  auto s_full = [&](int s) { return b0 + 8 * (2 * NS + s); };
  auto o_full = [&](int s) { return b0 + 8 * (2 * NS + 2 + s); };
  auto q_full = [&](int s) { return b0 + 8 * (2 * NS + 4 + s); };
  auto p_full = [&](int s, int half) { return b0 + 8 * (2 * NS + 6 + 2 * s + half); };
  const uint32_t fix = b0 + 8 * (2 * NS + 10), done = fix + 8;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      bar_init(full(s), 1);
      bar_init(empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(s_full(s), 1);
      bar_init(p_full(s, 0), 4);
      bar_init(p_full(s, 1), 4);
      bar_init(o_full(s), 1);
      bar_init(q_full(s), 4);
    }
    bar_init(fix, 1);
    bar_init(done, 1);
    gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (wid == 9) tmem_alloc(smem_u32(&tmem_base), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  pdl_trigger();
  const RowsTotals tot = rows_totals(a);
  int64_t x = cta_first_tile(tot.all, a.nc, blockIdx.x);
  const int64_t x_end = cta_first_tile(tot.all, a.nc, blockIdx.x + 1);
  bool first_of_cta = true;

  if (wid >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
  if (wid == 8) {  // ---------------------------------------------------------------- loads
    int slot = 0;
    uint32_t round = 0, fix_phase = 0;
    bool ok = true;
    int pend_slot = -1, pend_row = 0;  // a V tile whose rows from pend_row on are still to be cleared
    auto clear_pending = [&]() {
      if (pend_slot < 0) return true;
      if (!bar_wait(fix, fix_phase, &gave_up)) return false;
      fix_phase ^= 1;
      const uint32_t dst = ring + pend_slot * Sh::kTile;
      const int per = (kTcKeys - pend_row) * 8;
      for (int j = lane; j < per * PANELS; j += 32) {
        const int p = j / per, q = j - p * per;
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + p * kTcKeys * 128 + pend_row * 128 + q * 16), "r"(0)
                     : "memory");
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(full(pend_slot));
      pend_slot = -1;
      return true;
    };
    while (x < x_end && ok) {
      const RowsSeg s = rows_find(a, tot, x);
      const int64_t t0 = x - s.first, t1 = min64(s.first + s.tiles, x_end) - s.first;
      const int cnt = int(t1 - t0);
      const int seg_rows = s.own ? a.m * a.group : a.rows;
      const int lag = seg_rows - s.p * kTcRows > 128 ? 1 : 2;
      const CUtensorMap* mk = s.own ? &maps.ko : &maps.k;
      const CUtensorMap* mv = s.own ? &maps.vo : &maps.v;
      const int plane = s.own ? s.b * a.hkv + s.h : s.h;
      const int64_t len = s.own ? own_tokens(a, s.b) : a.n;
      for (int i = 0; i < cnt + lag && ok; ++i) {
#pragma unroll
        for (int kv = 1; kv >= 0; --kv) {  // V of tile i - lag, then K of tile i: the order of their use
          if (kv ? (!PV || i < lag) : i >= cnt) continue;
          const int64_t k0 = (t0 + (kv ? i - lag : i)) * kTcKeys;
          // rows of V past a sequence's end hold anything (0 * NaN is NaN): cleared before the product sees them, once the
          // copy has landed; meanwhile the next copies start, as long as none has to wait.  Past the prefix's end the
          // tensor map ends, so the copy itself fills zeros.
          const bool clear = kv && s.own && k0 + kTcKeys > len;
          if ((clear || !bar_done(empty(slot), (round & 1) ^ 1)) && !(ok = clear_pending())) break;
          if (!(ok = bar_wait(empty(slot), (round & 1) ^ 1, &gave_up))) break;
          const uint32_t dst = ring + slot * Sh::kTile;
          const uint32_t bar = clear ? fix : full(slot);
          if (lane == 0) {
            bar_expect(bar, Sh::kTile);
#pragma unroll
            for (int p = 0; p < PANELS; ++p)
              tma_load(dst + p * kTcKeys * 128, kv ? mv : mk, bar, p * 64, int(k0), plane);
          }
          if (clear) {
            pend_slot = slot;
            pend_row = int(len - k0);
          }
          if (++slot == NS) {
            slot = 0;
            ++round;
          }
        }
      }
      x = s.first + t1;
    }
    if (ok) clear_pending();
    // copies in flight when a wait gave up: let them land before the CTA's shared memory goes away
    if (gave_up) {
      int never = 0;
      for (int q = 0; q < NS; ++q) {
        const uint32_t r = q < slot ? round : round - 1;  // the slot's last use
        if (q < slot || round > 0) bar_wait(full(q), r & 1, &never);
      }
    }
  } else if (wid == 9) {  // ---------------------------------------------------------------- products
    int slot = 0;
    uint32_t round = 0;
    uint32_t p_phase[2] = {0, 0}, q_phase = 0;
    bool ok = true;
    constexpr uint32_t id_s = mma_idesc(kTcKeys, false), id_o = mma_idesc(D, true);
    while (x < x_end && ok) {
      const RowsSeg s = rows_find(a, tot, x);
      const int64_t t0 = x - s.first, t1 = min64(s.first + s.tiles, x_end) - s.first;
      const int cnt = int(t1 - t0);
      const int seg_rows = s.own ? a.m * a.group : a.rows;
      const bool both = seg_rows - s.p * kTcRows > 128;  // each stream its own rows
      const int lag = both ? 1 : 2;
      for (int st = 0; st < 2 && ok; ++st) ok = bar_wait(q_full(st), q_phase, &gave_up);
      q_phase ^= 1;
      if (!both && cnt == 1 && lane == 0) bar_arrive(o_full(1));  // stream 1 has no tile: nothing to wait for
      for (int i = 0; i < cnt + lag && ok; ++i) {
        const bool has_o = i >= lag, has_s = i < cnt;
        const int s_lo = both ? 0 : (i & 1), s_hi = both ? 1 : (i & 1);
        int v_slot = 0, k_slot = 0;
        if (PV && has_o) {
          v_slot = slot;
          ok = bar_wait(full(slot), round & 1, &gave_up);
          if (++slot == NS) {
            slot = 0;
            ++round;
          }
        }
        if (has_s && ok) {
          k_slot = slot;
          ok = bar_wait(full(slot), round & 1, &gave_up);
          if (++slot == NS) {
            slot = 0;
            ++round;
          }
        }
        for (int st = s_lo; st <= s_hi && ok; ++st) {
          const uint32_t ts = tm + st * 128, to = tm + 256 + st * D;
          if (has_o) {
            // the weights come in two halves of 64 keys: the products of the first run under the exponentials of the second
            const uint32_t v = ring + v_slot * Sh::kTile;
            const bool fresh = i == lag + (both ? 0 : (i & 1));  // the stream's first tile of the segment
#pragma unroll
            for (int half = 0; half < (PV ? 2 : 1); ++half) {
              if (!(ok = bar_wait(p_full(st, half), p_phase[st], &gave_up))) break;
              tc_fence_after();
              if (PV && lane == 0) {
#pragma unroll
                for (int k = half * 4; k < half * 4 + 4; ++k)
#pragma unroll
                  for (int part = 0; part < 2; ++part)
                    mma_ts(to, ts + (k / 2) * 32 + part * 16 + (k & 1) * 8, mma_desc(v + k * 2048, kTcKeys * 128), id_o,
                           !fresh || part || k);
              }
            }
            p_phase[st] ^= 1;
            if (!ok) break;
            if (PV && lane == 0) {
              if (st == s_hi) mma_commit(empty(v_slot));
              if (i + (both ? 1 : 2) >= cnt + lag) mma_commit(o_full(st));
            }
          }
          tc_fence_after();
          if (lane == 0) {
            if (has_s) {
              const uint32_t k = ring + k_slot * Sh::kTile;
#pragma unroll
              for (int e = 0; e < D / 16; ++e) {
                const uint32_t off = (e / 4) * (kTcKeys * 128) + (e % 4) * 32;
                mma_ss(ts, mma_desc(q_sm[st] + off, 16), mma_desc(k + off, 16), id_s, e > 0);
              }
              if (st == s_hi) mma_commit(empty(k_slot));
              mma_commit(s_full(st));
            }
          }
          __syncwarp();
        }
      }
      x = s.first + t1;
    }
    // nothing of the tensor pipe may be in flight when tensor memory is given back
    int never = 0;
    if (lane == 0) mma_commit(done);
    __syncwarp();
    bar_wait(done, 0, &never);
  } else if (wid == 10) {
    if (blockIdx.x == 0) rows_publish(a, tot);
  }
  } else {  // ---------------------------------------------------------------- the streams' rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    const int st = wid >> 2, row = tid & 127, wrow = (wid & 3) * 32;
    const uint32_t lane_base = uint32_t(wrow) << 16;
    const uint32_t ts = tm + lane_base + st * 128, to = tm + lane_base + 256 + st * D;
    const float c2 = a.scale * 1.4426950408889634f;  // weights as powers of two
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    while (x < x_end && ok) {
      const RowsSeg s = rows_find(a, tot, x);
      const int64_t t0 = x - s.first, t1 = min64(s.first + s.tiles, x_end) - s.first;
      const int cnt = int(t1 - t0);
      const int seg_rows = s.own ? a.m * a.group : a.rows;
      const int blk = s.p * kTcRows;
      const bool both = seg_rows - blk > 128;
      const int r0 = blk + (both ? st * 128 : 0);  // the stream's first row
      const int nrows = min(128, seg_rows - r0);
      const int row_off = s.own ? s.b * a.m * a.group : 0;
      constexpr int CH = D / 8, RP = 128 / CH;  // 16-byte pieces of a row, rows per pass of the stream's threads
      {
        const int c = row % CH, rq = row / CH;
        const __nv_bfloat16* Qp = static_cast<const __nv_bfloat16*>(a.Q) + c * 8;
        const uint32_t dst = q_sm[st] + (c / 8) * (128 * 128);
#pragma unroll
        for (int g = 0; g < CH; g += 8) {  // eight loads in flight
          uint4 v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int r = (g + q) * RP + rq;
            v[q] = r < nrows ? *reinterpret_cast<const uint4*>(Qp + row_index(a, s.h, row_off + r0 + r) * D)
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
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(q_full(st));
      const int64_t len = s.own ? own_tokens(a, s.b) : a.n;
      const int64_t lim = row >= nrows ? 0 : (s.own ? own_limit(a, len, r0 + row) : prefix_limit(a, r0 + row));
      const bool active = wrow < nrows;  // a warp of padding rows leaves its weights alone: they reach no valid row
      float m_ref = -INFINITY, l_run = 0.f;
      const int step = both ? 1 : 2, i0 = both ? 0 : st;
      for (int i = i0; i < cnt; i += step) {
        if (!(ok = bar_wait(s_full(st), s_phase, &gave_up))) break;
        s_phase ^= 1;
        tc_fence_after();
        if (active) {
          float sv[kTcKeys];
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld32(ts + 32 * j, sv + 32 * j);
          tmem_wait_ld();
          const int64_t left = lim - (t0 + i) * kTcKeys;
          if (__any_sync(0xffffffffu, left < kTcKeys)) {
            const int n_vis = left < 0 ? 0 : (left > kTcKeys ? kTcKeys : int(left));
#pragma unroll
            for (int j = 0; j < kTcKeys; ++j)
              if (j >= n_vis) sv[j] = -INFINITY;
          }
          float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int j = 4; j + 8 <= kTcKeys; j += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], sv[j + q], sv[j + 4 + q]);
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], sv[kTcKeys - 4 + q]);
          const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
          const bool grow = m_new > m_ref + kLazyMax || (m_ref == -INFINITY && m_new > -INFINITY);
          if (__any_sync(0xffffffffu, grow)) {
            const float up = grow ? m_new : m_ref;
            const float sc = m_ref == -INFINITY ? 0.f : ex2(m_ref - up);
            if (PV && i != i0) {
              // l > 0 is not needed: a row without weights so far has O = 0 (or NaN from NaN)
#pragma unroll
              for (int j = 0; j < D / 32; ++j) {
                float o[32];
                tmem_ld32(to + 32 * j, o);
                tmem_wait_ld();
                if (grow) {
#pragma unroll
                  for (int q = 0; q < 32; ++q) o[q] = m_ref == -INFINITY ? 0.f : o[q] * sc;
                }
                tmem_st32(to + 32 * j, reinterpret_cast<const uint32_t*>(o));
              }
            }
            if (grow) {
              l_run *= sc;
              m_ref = up;
            }
          }
          const float mb = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t cc = pair(c2, c2), mm = pair(-mb, -mb), minus = pair(-1.f, -1.f);
          uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[32];  // 32 keys: their hi parts, then their lo parts
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              float e0, e1;
              unpair(fma2(pair(sv[32 * j + 2 * q], sv[32 * j + 2 * q + 1]), cc, mm), &e0, &e1);
              const uint64_t p = pair(ex2(e0), ex2(e1));
              sum[q & 1] = add2(sum[q & 1], p);
              if (PV) {
                float p0, p1;
                unpair(p, &p0, &p1);
                w[q] = pack_bf16(p0, p1);
                unpair(fma2(pair(__uint_as_float(w[q] << 16), __uint_as_float(w[q] & 0xffff0000u)), minus, p), &p0, &p1);
                w[16 + q] = pack_bf16(p0, p1);
              }
            }
            if (PV) {
              tmem_st32(ts + 32 * j, w);
              if (j & 1) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(p_full(st, j >> 1));
              }
            }
          }
          float s0, s1;
          unpair(add2(sum[0], sum[1]), &s0, &s1);
          l_run += s0 + s1;
        }
        if (!PV || !active) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(p_full(st, 0));
            if (PV) bar_arrive(p_full(st, 1));
          }
        }
      }
      if (!ok) break;
      const bool any = i0 < cnt;  // a single tile leaves stream 1 without work
      if (PV || !any) {  // also without work: the stream stays within one segment of the products' warp
        if (!(ok = bar_wait(o_full(st), o_phase, &gave_up))) break;
        o_phase ^= 1;
        tc_fence_after();
      }
      // the segment's share of this CTA: a partial per stream, or the result where this CTA's streams hold all tiles
      const bool whole = !a.has_own && both && x == s.first && t1 == s.tiles;
      if (active) {
        const int64_t pr = part_row(a, blockIdx.x, s.own, s.id, first_of_cta) +
                           (both ? st * 128 : st * ((s.own ? a.ro : a.rp) / 2)) + row;
        const int64_t ri = row < nrows ? row_index(a, s.h, row_off + r0 + row) : 0;
        float inv = 1.f;
        if (row < nrows) {
          if (whole) {
            inv = l_run == 0.f ? 0.f : 1.f / l_run;
            if (a.lse) a.lse[ri] = l_run > 0.f ? (m_ref + log2f(l_run)) * 0.6931471805599453f : (l_run == 0.f ? -INFINITY : l_run);
          } else {
            a.part_ml[pr] = make_float2(m_ref, l_run);
          }
        }
        if (PV && any) {
          float* dst = whole ? a.O + ri * D : a.part + pr * D;
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            float o[32];
            tmem_ld32(to + 32 * j, o);
            tmem_wait_ld();
            if (row < nrows) {
#pragma unroll
              for (int q = 0; q < 32; q += 4)
                *reinterpret_cast<float4*>(dst + 32 * j + q) =
                    make_float4(o[q] * inv, o[q + 1] * inv, o[q + 2] * inv, o[q + 3] * inv);
            }
          }
        }
      }
      tc_fence_before();
      first_of_cta = false;
      x = s.first + t1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (gave_up && tid == 0) raise_status(a.status, ZHA_ERR_TIMEOUT);
  if (wid == 9) tmem_free(tm, 512);
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

template <int D, bool PV> cudaError_t run_tc(const RowsArgs& a, const TcMaps& maps, cudaStream_t st) {
  const cudaError_t e = allow_smem(rows_tc_kernel<D, PV>, TcShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  rows_tc_kernel<D, PV><<<a.nc, kTcThreads, TcShape<D>::kSmem, st>>>(a, maps);
  return cudaGetLastError();
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
  if (a.O) return d == 128 ? run_tc<128, true>(a, maps, st) : run_tc<64, true>(a, maps, st);
  return d == 128 ? run_tc<128, false>(a, maps, st) : run_tc<64, false>(a, maps, st);
}

// At most one CTA per SM, and none without a tile.  A row block of at most 128 rows has a partial per stream.
void tc_plan(int hkv, int64_t B, int64_t rows, int64_t mg, int64_t n, int64_t ld_own, RowsPlan* p) {
  p->kt = kTcKeys;
  p->rb = kTcRows;
  p->pp = int((rows + kTcRows - 1) / kTcRows);
  p->po = ld_own > 0 ? int((mg + kTcRows - 1) / kTcRows) : 0;
  p->rp = rows > 128 ? kTcRows : int(2 * rows);
  p->ro = mg > 128 ? kTcRows : int(2 * mg);
  const double tiles = double(hkv) * p->pp * double((n + kTcKeys - 1) / kTcKeys) +
                       double(B) * hkv * p->po * double((ld_own + kTcKeys - 1) / kTcKeys);
  p->nc = tiles < 1 ? 1 : (tiles < 148 ? int(tiles) : 148);
}

}  // namespace zha
