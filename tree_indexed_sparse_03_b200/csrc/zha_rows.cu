// Many query rows over one KV cache on the CUDA cores (fp32 configurations),
// the join of the partials, and the column sums of the softmax weights.
// The work split is described in zha_rows.cuh.
#include "zha_rows.cuh"

namespace zha {

constexpr int kRowsThreads = 128;
constexpr int kRowsKeys = 64;  // keys per tile
constexpr int kWeightsCtas = 148 * 4;  // CTAs that the weights pass splits its rows up to

// ------------------------------------------------------------------ attention, CUDA cores
// One CTA: RB = 8 * RT rows against tiles of 64 keys.  A half-warp owns RT rows: for S = Q K^T each lane holds RT
// rows x 4 keys (key = lane + 16 j), so a row's maximum and sum are shuffles within the half-warp; for O += P V each
// lane holds the same RT rows x d/16 columns, P passed through shared memory within the warp.  Rows of shared memory
// are padded by 16 bytes, so 16-byte reads of 8 consecutive rows meet no bank conflict.  Per 4 dimensions a lane
// does 16 RT FMAs on RT + 4 16-byte reads: the FMA pipe bounds it for RT >= 4 (16 sequences x 4 heads behind 16K
// tokens, d = 128: 91 us, 24 TFLOP/s), shared-memory reads and HBM for RT = 1 (8 rows over 64K tokens: 110 us, 2.4
// TB/s; with two pieces of K and V in flight per thread instead of sixteen 162 us).
template <typename T, int D, int RT>
__global__ void __launch_bounds__(kRowsThreads) rows_scalar_kernel(RowsArgs a) {
  constexpr int RB = 8 * RT, LD = D + 4, PLD = kRowsKeys + 4, CT = D / 16;
  constexpr int EPC = 16 / sizeof(T), CPR = D / EPC;  // elements per 16-byte chunk, chunks per row
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;
  float* sk = sq + RB * LD;
  float* sv = sk + kRowsKeys * LD;
  float* sp = sv + kRowsKeys * LD;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int half = wid * 2 + (lane >> 4), l16 = lane & 15;
  const float c2 = a.scale * 1.4426950408889634f;  // weights as powers of two
  pdl_trigger();
  pdl_wait();
  const RowsTotals tot = rows_totals(a);
  if (blockIdx.x == 0 && wid == 0) rows_publish(a, tot);
  const int x_begin = tot.sh.begin(blockIdx.x), x_end = tot.sh.begin(blockIdx.x + 1);
  for (int x = x_begin; x < x_end;) {
    const RowsSeg s = rows_find(a, tot, x);
    const int t_begin = x - s.first, t_end = min(s.first + s.tiles, x_end) - s.first;
    x = s.next;
    if (t_begin >= t_end) continue;
    const int seg_rows = s.own ? a.m * a.group : a.rows;
    const int r0 = s.p * RB;
    const int nrows = min(RB, seg_rows - r0);
    const int row_off = s.own ? s.b * a.m * a.group : 0;  // the sequence's first row of the head
    const int64_t len = s.own ? own_tokens(a, s.b) : a.n;
    const T* Kh = s.own ? static_cast<const T*>(a.Ko) + (int64_t(s.b) * a.hkv + s.h) * a.ld_own * D
                        : static_cast<const T*>(a.K) + int64_t(s.h) * a.ld * D;
    const T* Vh = s.own ? static_cast<const T*>(a.Vo) + (int64_t(s.b) * a.hkv + s.h) * a.ld_own * D
                        : (a.V ? static_cast<const T*>(a.V) + int64_t(s.h) * a.ld * D : nullptr);
    __syncthreads();
    for (int i = tid; i < RB * CPR; i += kRowsThreads) {
      const int r = i / CPR, c = i % CPR;
      float v[EPC];
#pragma unroll
      for (int e = 0; e < EPC; ++e) v[e] = 0.f;
      if (r < nrows)
        unpack16<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.Q) +
                                                    row_index(a, s.h, row_off + r0 + r) * D + c * EPC), v);
#pragma unroll
      for (int e = 0; e < EPC; e += 4)
        *reinterpret_cast<float4*>(sq + r * LD + c * EPC + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    }
    int64_t lim[RT];
    float m_run[RT], l_run[RT], o[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = r0 + half * RT + i;
      lim[i] = r >= seg_rows ? 0 : (s.own ? own_limit(a, len, r) : prefix_limit(a, r));
      m_run[i] = -INFINITY;
      l_run[i] = 0.f;
#pragma unroll
      for (int j = 0; j < CT; ++j) o[i][j] = 0.f;
    }
    for (int t = t_begin; t < t_end; ++t) {
      const int64_t k0 = int64_t(t) * kRowsKeys;
      __syncthreads();
      constexpr int G = RT < 8 ? 8 : 4;  // 16-byte pieces of K and of V in flight per thread (RT = 8: the registers are needed)
#pragma unroll 1
      for (int i0 = tid; i0 < kRowsKeys * CPR; i0 += G * kRowsThreads) {
        uint4 kr[G], vr[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int i = i0 + g * kRowsThreads, r = i / CPR, c = i % CPR;
          kr[g] = vr[g] = make_uint4(0, 0, 0, 0);  // keys past the range: zeros, never what lies there
          if (k0 + r < len) {
            kr[g] = ldg_stream(Kh + (k0 + r) * D + c * EPC);
            if (Vh) vr[g] = ldg_stream(Vh + (k0 + r) * D + c * EPC);
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int i = i0 + g * kRowsThreads, r = i / CPR, c = i % CPR;
          float k[EPC], v[EPC];
          unpack16<T>(kr[g], k);
          unpack16<T>(vr[g], v);
#pragma unroll
          for (int e = 0; e < EPC; e += 4) {
            *reinterpret_cast<float4*>(sk + r * LD + c * EPC + e) = make_float4(k[e], k[e + 1], k[e + 2], k[e + 3]);
            if (Vh) *reinterpret_cast<float4*>(sv + r * LD + c * EPC + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
      }
      __syncthreads();
      float acc[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll 4
      for (int e = 0; e < D; e += 4) {
        float4 kv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(sk + (l16 + 16 * j) * LD + e);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float4 qv = *reinterpret_cast<const float4*>(sq + (half * RT + i) * LD + e);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][j] = fmaf(qv.x, kv[j].x, acc[i][j]);
            acc[i][j] = fmaf(qv.y, kv[j].y, acc[i][j]);
            acc[i][j] = fmaf(qv.z, kv[j].z, acc[i][j]);
            acc[i][j] = fmaf(qv.w, kv[j].w, acc[i][j]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float mx = m_run[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = k0 + l16 + 16 * j < lim[i] ? acc[i][j] * c2 : -INFINITY;
          mx = fmaxf(mx, acc[i][j]);
        }
        if (a.logits && r0 + half * RT + i < seg_rows) {
          float* lg = a.logits + (int64_t(s.h) * a.rows + r0 + half * RT + i) * a.ld_logits + k0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (k0 + l16 + 16 * j < a.n) __stcg(lg + l16 + 16 * j, acc[i][j]);
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float base = mx == -INFINITY ? 0.f : mx;  // a row that sees nothing yet: every weight 2^-inf = 0
        const float sc = exp2f(m_run[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(acc[i][j] - base);
          sum += p;
          if (Vh) sp[(half * RT + i) * PLD + l16 + 16 * j] = p;
        }
        l_run[i] = fmaf(l_run[i], sc, sum);
        m_run[i] = mx;
#pragma unroll
        for (int j = 0; j < CT; ++j) o[i][j] *= sc;
      }
      if (Vh) {
        __syncwarp();
#pragma unroll 2
        for (int k = 0; k < kRowsKeys; k += 4) {
          float4 pv[RT];
#pragma unroll
          for (int i = 0; i < RT; ++i) pv[i] = *reinterpret_cast<const float4*>(sp + (half * RT + i) * PLD + k);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            float vv[CT];
#pragma unroll
            for (int j = 0; j < CT; j += 4) {  // columns l16*4 + 64*(j/4): 16 lanes read 256 contiguous bytes
              const float4 v4 = *reinterpret_cast<const float4*>(sv + (k + kk) * LD + l16 * 4 + 16 * j);
              vv[j] = v4.x;
              vv[j + 1] = v4.y;
              vv[j + 2] = v4.z;
              vv[j + 3] = v4.w;
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              const float p = kk == 0 ? pv[i].x : (kk == 1 ? pv[i].y : (kk == 2 ? pv[i].z : pv[i].w));
#pragma unroll
              for (int j = 0; j < CT; ++j) o[i][j] = fmaf(p, vv[j], o[i][j]);
            }
          }
        }
        __syncwarp();
      }
    }
    // the segment's share of this CTA: a partial, or the row's result where the CTA holds the whole segment
    const bool whole = !a.has_own && t_begin == 0 && t_end == s.tiles;
    const int64_t slot = part_row(a, blockIdx.x, s.own, s.id, x_begin < s.first);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int rl = half * RT + i;
      float l = l_run[i];
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      if (rl < nrows) {
        const int64_t ri = row_index(a, s.h, row_off + r0 + rl);
        if (l16 == 0) {
          if (!whole) a.part_ml[slot + rl] = make_float2(m_run[i], l);
          else if (a.lse) a.lse[ri] = l > 0.f ? (m_run[i] + log2f(l)) * 0.6931471805599453f : (l == 0.f ? -INFINITY : l);
        }
        if (a.O) {
          const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
          float* dst = whole ? a.O + ri * D : a.part + (slot + rl) * D;
#pragma unroll
          for (int j = 0; j < CT; j += 4)
            *reinterpret_cast<float4*>(dst + l16 * 4 + 16 * j) =
                make_float4(o[i][j] * inv, o[i][j + 1] * inv, o[i][j + 2] * inv, o[i][j + 3] * inv);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ join of the partials
// o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the CTAs that touched the
// row's segments, in CTA order (prefix first); W warps per row take strided
// partials and are joined in warp order, so the result does not depend on timing.
template <int D, int W>
__global__ void __launch_bounds__(256) rows_combine_kernel(RowsArgs a) {
  constexpr int EL = D / 32;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int h = blockIdx.y, r = int(blockIdx.x) * (8 / W) + wid / W;  // KV head, row
  const int w = wid % W;
  const bool live = r < a.rows;
  pdl_trigger();
  pdl_wait();
  Shares sh;
  sh.set(a.plan[0], a.nc);
  // the row's prefix partials: CTAs c_lo[0] .. + cnt[0] - 1, its own ones likewise
  int c_lo[2] = {0, 0}, cnt[2] = {0, 0}, id[2], rl[2], first[2];
  bool direct = false;
  if (live) {
    const int p = r >> a.rb_log, base = a.plan[3 + p], tiles = a.plan[4 + p] - base - a.extra;
    rl[0] = r - (p << a.rb_log);
    first[0] = h * a.plan[1] + base;
    id[0] = h * a.pp + p;
    if (tiles > 0) {
      c_lo[0] = sh.owner(first[0]);
      cnt[0] = sh.owner(first[0] + tiles - 1) - c_lo[0] + 1;
      direct = !a.has_own && cnt[0] == 1;  // written by its CTA
    }
    if (a.has_own) {
      const int mg = a.m * a.group, b = r / mg, rs = r - b * mg, q = rs >> a.rb_log;
      const int ob = a.plan[4 + a.pp + b], span = a.plan[5 + a.pp + b] - ob, u = h * a.po + q;
      rl[1] = rs - (q << a.rb_log);
      first[1] = a.plan[2] + ob * (a.hkv * a.po) + u * span;
      id[1] = a.hkv * a.pp + b * a.hkv * a.po + u;
      if (span > 0) {
        c_lo[1] = sh.owner(first[1]);
        cnt[1] = sh.owner(first[1] + span - a.extra - 1) - c_lo[1] + 1;
      }
    }
  }
  const int total = direct ? 0 : cnt[0] + cnt[1];
  // a warp takes a contiguous run, 32 partials at a time: their scales lane by lane, their rows four in flight
  const int run = (total + W - 1) / W, q_end = min(total, (w + 1) * run);
  float M = -INFINITY, L = 0.f, o[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) o[e] = 0.f;
  for (int q0 = w * run; q0 < q_end; q0 += 32) {
    const int q = q0 + lane, have = min(32, q_end - q0);
    int64_t pr = 0;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < have) {
      const int k = q >= cnt[0], c = c_lo[k] + (k ? q - cnt[0] : q);
      pr = part_row(a, c, k, id[k], sh.begin(c) < first[k]) + rl[k];
      ml = __ldcg(a.part_ml + pr);
    }
    float mn = fmaxf(M, ml.x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    const float base = mn == -INFINITY ? 0.f : mn;
    const bool none = ml.x == -INFINITY && ml.y == 0.f;  // nothing of this share is visible to the row
    const float sc = none ? 0.f : exp2f(ml.x - base), keep = exp2f(M - base);
    float l = none ? 0.f : ml.y * sc;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    L = L * keep + l;
#pragma unroll
    for (int e = 0; e < EL; ++e) o[e] *= keep;
    M = mn;
    if (a.O) {
#pragma unroll 4
      for (int j = 0; j < have; ++j) {
        const float s = __shfl_sync(0xffffffffu, sc, j);
        const int64_t row = __shfl_sync(0xffffffffu, pr, j);
        const bool skip = __shfl_sync(0xffffffffu, int(none), j);
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          const float v = __ldcg(a.part + row * D + lane + 32 * e);
          if (!skip) o[e] = fmaf(v, s, o[e]);
        }
      }
    }
  }
  __shared__ float jm[8], jl[8], jo[8][D];
  if (W > 1) {
    if (lane == 0) {
      jm[wid] = M;
      jl[wid] = L;
    }
#pragma unroll
    for (int e = 0; e < EL; ++e) jo[wid][lane + 32 * e] = o[e];
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int q = 1; q < W; ++q) {
        const float m_s = jm[wid + q];
        if (m_s == -INFINITY && jl[wid + q] == 0.f) continue;
        const float mn = fmaxf(M, m_s), s0 = M == -INFINITY ? 0.f : exp2f(M - mn), s1 = exp2f(m_s - mn);
        L = L * s0 + jl[wid + q] * s1;
#pragma unroll
        for (int e = 0; e < EL; ++e) o[e] = o[e] * s0 + jo[wid + q][lane + 32 * e] * s1;
        M = mn;
      }
    }
  }
  if (live && w == 0 && !direct) {
    const int64_t ri = row_index(a, h, r);
    if (a.O) {
      const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
      for (int e = 0; e < EL; ++e) a.O[ri * D + lane + 32 * e] = o[e] * inv;
    }
    if (a.lse && lane == 0) a.lse[ri] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : (L == 0.f ? -INFINITY : L);
  }
}

// ------------------------------------------------------------------ column sums of the weights, CUDA cores
// acc_out[h][k] = acc_in[h][k] + sum over rows of 2^(s c - lse): one CTA per (64 keys, KV head, row split); a lane
// holds RT rows x 4 keys of S as above and sums over its rows; the eight half-warps are joined in order.  230 rows x
// 4 heads over 9,000 tokens, causal, d = 128: 182 us with the attention before it, 193 with the keys loaded one
// piece at a time.

// ROWS padded rows of shared memory from row(r) (NULL: zeros), all 128 threads, G 16-byte pieces in flight per
// thread.
template <typename T, int D, int ROWS, typename F> __device__ __forceinline__ void fill_rows(float* dst, F row) {
  constexpr int EPC = 16 / sizeof(T), CPR = D / EPC, LD = D + 4, N = ROWS * CPR / kRowsThreads, G = N < 8 ? N : 8;
  static_assert(N * kRowsThreads == ROWS * CPR && N % G == 0, "whole rounds");
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < ROWS * CPR; i0 += G * kRowsThreads) {
    uint4 v[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int i = i0 + g * kRowsThreads;
      const T* p = row(i / CPR);
      v[g] = p ? ldg_stream(p + i % CPR * EPC) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int i = i0 + g * kRowsThreads;
      float f[EPC];
      unpack16<T>(v[g], f);
#pragma unroll
      for (int e = 0; e < EPC; e += 4)
        *reinterpret_cast<float4*>(dst + i / CPR * LD + i % CPR * EPC + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    }
  }
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kRowsThreads) weights_scalar_kernel(WeightsArgs a) {
  constexpr int RB = 8 * RT, LD = D + 4;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;
  float* sk = sq + RB * LD;
  float* sl = sk + kRowsKeys * LD;  // lse of the block's rows, in powers of two
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int half = wid * 2 + (lane >> 4), l16 = lane & 15;
  const float c2 = a.scale * 1.4426950408889634f;
  const int64_t k0 = int64_t(blockIdx.x) * kRowsKeys;
  const int h = blockIdx.y;
  pdl_trigger();
  pdl_wait();
  const T* Kh = static_cast<const T*>(a.K) + int64_t(h) * a.ld * D;
  fill_rows<T, D, kRowsKeys>(sk, [&](int r) { return k0 + r < a.n ? Kh + (k0 + r) * D : nullptr; });
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  const int rend = int(min64(a.rows, int64_t(blockIdx.z + 1) * a.rows_per_split));
  int rbeg = int(int64_t(blockIdx.z) * a.rows_per_split);
  if (a.causal) {  // rows before the first that sees this tile's first key
    const int first = int(max64(0, k0 - (a.n - a.m))) * a.group;
    if (first > rbeg) rbeg = first / RB * RB;
  }
  for (int r0 = rbeg; r0 < rend; r0 += RB) {
    __syncthreads();
    auto q_row = [&](int rr) {
      const int t = rr / a.group;
      return int64_t(t) * a.hq + h * a.group + (rr - t * a.group);
    };
    fill_rows<T, D, RB>(sq, [&](int r) {
      return r0 + r < rend ? static_cast<const T*>(a.Q) + q_row(r0 + r) * D : nullptr;
    });
    if (tid < RB)  // no row: every weight 2^-inf = 0
      sl[tid] = r0 + tid < rend ? a.lse[q_row(r0 + tid)] * 1.4426950408889634f : INFINITY;
    __syncthreads();
    float acc[RT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
      float4 kv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(sk + (l16 + 16 * j) * LD + e);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const float4 qv = *reinterpret_cast<const float4*>(sq + (half * RT + i) * LD + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = fmaf(qv.x, kv[j].x, acc[i][j]);
          acc[i][j] = fmaf(qv.y, kv[j].y, acc[i][j]);
          acc[i][j] = fmaf(qv.z, kv[j].z, acc[i][j]);
          acc[i][j] = fmaf(qv.w, kv[j].w, acc[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int rr = r0 + half * RT + i;
      const int64_t lim = a.causal ? a.n - a.m + rr / a.group + 1 : a.n;
      const float ls = sl[half * RT + i];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k0 + l16 + 16 * j < lim) sum[j] += exp2f(fmaf(acc[i][j], c2, -ls));
    }
  }
  __syncthreads();
  float* red = sq;  // [8][64]
#pragma unroll
  for (int j = 0; j < 4; ++j) red[half * kRowsKeys + l16 + 16 * j] = sum[j];
  __syncthreads();
  if (tid < kRowsKeys && k0 + tid < a.n) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += red[q * kRowsKeys + tid];
    if (a.rsplit > 1) {
      a.sums[(int64_t(blockIdx.z) * a.hkv + h) * a.n + k0 + tid] = s;
    } else {
      a.acc_out[h * a.ld_acc_out + k0 + tid] = (a.acc_in ? a.acc_in[h * a.ld_acc_in + k0 + tid] : 0.f) + s;
    }
  }
}

// acc_out = acc_in + the row splits' sums, in split order.
__global__ void __launch_bounds__(256) weights_join_kernel(WeightsArgs a) {
  const int64_t k = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int h = blockIdx.y;
  pdl_wait();
  if (k >= a.n) return;
  float s = 0.f;
  for (int z = 0; z < a.rsplit; ++z) s += a.sums[(int64_t(z) * a.hkv + h) * a.n + k];
  a.acc_out[h * a.ld_acc_out + k] = (a.acc_in ? a.acc_in[h * a.ld_acc_in + k] : 0.f) + s;
}

// acc_out = acc_in + the weights of the kept logits: four keys per thread, all rows' logits in flight.  Bound by the
// logits' way through L2.
__global__ void __launch_bounds__(256) weights_logits_kernel(WeightsArgs a) {
  __shared__ float lse2[kLogitRows];
  const int h = blockIdx.y;
  const int64_t k = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  pdl_wait();
  const bool failed = a.status && __ldcg(a.status) != 0;  // a wait ran out: the logits may not be these queries'
  if (threadIdx.x < a.rows) {
    const int t = threadIdx.x / a.group;
    lse2[threadIdx.x] = a.lse[int64_t(t) * a.hq + h * a.group + (threadIdx.x - t * a.group)] * 1.4426950408889634f;
  }
  __syncthreads();
  if (k >= a.n || failed) return;
  const float* lg = a.logits + int64_t(h) * a.rows * a.ld_logits + k;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int r = 0; r < a.rows; ++r) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(lg + r * a.ld_logits));
    s[0] += exp2f(t.x - lse2[r]);
    s[1] += exp2f(t.y - lse2[r]);
    s[2] += exp2f(t.z - lse2[r]);
    s[3] += exp2f(t.w - lse2[r]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (k + e < a.n) a.acc_out[h * a.ld_acc_out + k + e] = (a.acc_in ? a.acc_in[h * a.ld_acc_in + k + e] : 0.f) + s[e];
}

// Sums in place, last: acc_out = the staged sums, unless a wait of the tensor-core kernels before has run out (some CTAs
// may then have left without theirs).
__global__ void __launch_bounds__(256) weights_commit_kernel(WeightsArgs a, float* acc_out, int64_t ld_acc_out) {
  const int h = blockIdx.y;
  const int64_t k0 = int64_t(blockIdx.x) * 1024 + threadIdx.x;
  pdl_wait();
  if (__ldcg(a.status) != 0) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t k = k0 + 256 * e;
    if (k < a.n) acc_out[h * ld_acc_out + k] = __ldcg(a.acc_out + h * a.ld_acc_out + k);
  }
}

// ------------------------------------------------------------------ host side
namespace {

// Rows per half-warp: few rows leave most of a larger block empty, more rows share each key read from shared memory.
int scalar_rt(int d, int64_t rows) { return rows <= 8 ? 1 : (d == 128 || rows <= 32 ? 4 : 8); }

size_t rows_smem(int d, int rt) {
  return size_t(8 * rt * (d + 4) + 2 * kRowsKeys * (d + 4) + 8 * rt * (kRowsKeys + 4)) * sizeof(float);
}

size_t weights_smem(int d, int rt) { return size_t(8 * rt * (d + 4) + kRowsKeys * (d + 4) + 8 * rt) * sizeof(float); }

template <typename T, int D, int RT> cudaError_t run_rows(const RowsArgs& a, cudaStream_t st) {
  const size_t sm = rows_smem(D, RT);
  cudaError_t e = allow_smem(rows_scalar_kernel<T, D, RT>, sm);
  if (e != cudaSuccess) return e;
  return launch_after(rows_scalar_kernel<T, D, RT>, dim3(a.nc), kRowsThreads, sm, st, a);
}

template <typename T, int D> cudaError_t run_rows_rt(const RowsArgs& a, cudaStream_t st) {
  switch (1 << a.rb_log >> 3) {
    case 1: return run_rows<T, D, 1>(a, st);
    case 8: if constexpr (D == 64) return run_rows<T, D, 8>(a, st);  // d = 128: registers and shared memory for half
    default: return run_rows<T, D, 4>(a, st);
  }
}

template <int D> cudaError_t run_combine(const RowsArgs& a, cudaStream_t st) {
  // few rows: eight warps share a row's partials (up to two per CTA); many rows have few partials each
  if (a.rows * a.hkv < 2048) return launch_after(rows_combine_kernel<D, 8>, dim3(a.rows, a.hkv), 256, 0, st, a);
  return launch_after(rows_combine_kernel<D, 1>, dim3((a.rows + 7) / 8, a.hkv), 256, 0, st, a);
}

template <typename T, int D, int RT> cudaError_t run_weights(const WeightsArgs& a, cudaStream_t st) {
  const size_t sm = weights_smem(D, RT);
  cudaError_t e = allow_smem(weights_scalar_kernel<T, D, RT>, sm);
  if (e != cudaSuccess) return e;
  const dim3 grid(unsigned((a.n + kRowsKeys - 1) / kRowsKeys), unsigned(a.hkv), unsigned(a.rsplit));
  return launch_after(weights_scalar_kernel<T, D, RT>, grid, kRowsThreads, sm, st, a);
}

template <typename T, int D> cudaError_t run_weights_rt(const WeightsArgs& a, cudaStream_t st) {
  switch (scalar_rt(D, a.rows)) {
    case 1: return run_weights<T, D, 1>(a, st);
    case 8: if constexpr (D == 64) return run_weights<T, D, 8>(a, st);
    default: return run_weights<T, D, 4>(a, st);
  }
}

}  // namespace

// CTAs (at most `most`, and no more than tiles) and partial rows of a plan whose row blocks and tiles are set.  Own
// caches are taken as long as they can be.
static void plan_parts(int hkv, int64_t B, int64_t n, int64_t ld_own, int most, RowsPlan* p) {
  const double pt = double((n + (1 << p->kt_log) - 1) >> p->kt_log), ot = double((ld_own + (1 << p->kt_log) - 1) >> p->kt_log);
  const double ps = double(hkv) * p->pp, os = double(B) * hkv * p->po;
  const double tiles = ps * pt + os * ot;
  p->places = tiles + (ps + os) * p->extra;
  p->nc = tiles < 1 ? 1 : (tiles < most ? int(tiles) : most);
  if (ld_own > 0) {
    p->part_own = (uint64_t(p->nc) + uint64_t(hkv) * p->pp) * p->rp;
    p->part_rows = p->part_own + (uint64_t(p->nc) + uint64_t(B) * hkv * p->po) * p->ro;
  } else {
    p->part_own = 0;
    p->part_rows = 2 * uint64_t(p->nc) * p->rp;
  }
  p->part_tmp = p->part_rows;
  p->part_rows += uint64_t(p->nc) * p->rt;
}

static void scalar_plan(int d, int rt, int hkv, int64_t B, int64_t rows, int64_t mg, int64_t n, int64_t ld_own,
                        RowsPlan* p) {
  const int rb = 8 * rt;
  p->rb_log = rt == 1 ? 3 : (rt == 4 ? 5 : 6);
  p->kt_log = 6;
  p->extra = 1;  // queries, first loads and the write-out of a segment take about as long as a tile
  p->pp = int((rows + rb - 1) / rb);
  p->po = ld_own > 0 ? int((mg + rb - 1) / rb) : 0;
  p->rp = int(rows < rb ? rows : rb);
  p->ro = int(mg < rb ? mg : rb);
  p->rt = 0;
  const int per_sm = int(220 * 1024 / (rows_smem(d, rt) + 1024));
  plan_parts(hkv, B, n, ld_own, 148 * (per_sm < 1 ? 1 : (per_sm > 4 ? 4 : per_sm)), p);
}

void rows_plan(int dtype, int d, int hkv, int group, int64_t B, int64_t m, int64_t n, int64_t ld_own, RowsPlan* p) {
  const int64_t rows = B * m * group;
  if (dtype == ZHA_BF16) {
    tc_plan(rows, m * group, ld_own, p);
    plan_parts(hkv, B, n, ld_own, 148, p);
  } else {
    scalar_plan(d, scalar_rt(d, rows), hkv, B, rows, m * group, n, ld_own, p);
  }
}

// Partial rows that cover every call with at most B sequences, m query tokens, n and ld_own tokens.  For one
// variant the plan's rows grow with each of them; smaller calls may take a variant of fewer rows per block.
uint64_t rows_part_bound(int dtype, int d, int hkv, int group, int64_t B, int64_t m, int64_t n, int64_t ld_own) {
  const int64_t rows = B * m * group, mg = m * group;
  uint64_t most = 0;
  for (int rt = 1; rt <= 8; rt = rt == 1 ? 4 : 2 * rt) {
    const int64_t cap = rt == 1 ? 8 : (rt == 4 && d == 64 ? 32 : rows);  // rows that take this variant
    if (dtype != ZHA_BF16 && rt > scalar_rt(d, rows)) break;
    for (int own = 0; own < 2; ++own) {
      RowsPlan p;
      if (dtype == ZHA_BF16) {
        tc_plan(rows, mg, own ? ld_own : 0, &p);
        plan_parts(hkv, B, n, own ? ld_own : 0, 148, &p);
      } else {
        scalar_plan(d, rt, hkv, min64(B, cap), min64(rows, cap), min64(mg, cap), n, own ? ld_own : 0, &p);
      }
      if (p.part_rows > most) most = p.part_rows;
    }
  }
  return most;
}

cudaError_t launch_rows(const RowsArgs& a, int dtype, int d, cudaStream_t st) {
  count_launches(2);
  cudaError_t e;
  if (dtype == ZHA_BF16) e = launch_rows_tc(a, d, st);
  else e = d == 128 ? run_rows_rt<float, 128>(a, st) : run_rows_rt<float, 64>(a, st);
  if (e != cudaSuccess) return e;
  return d == 128 ? run_combine<128>(a, st) : run_combine<64>(a, st);
}

void weights_plan(int dtype, int d, int hkv, int64_t rows, int64_t n, WeightsPlan* p) {
  if (dtype == ZHA_BF16) {
    p->rsplit = 1;
    p->rows_per_split = rows;
    p->sum_floats = weights_tc_floats() + uint64_t(hkv) * uint64_t(n);  // and the sums in place until they are complete
    p->places = double(hkv) * double((n + 255) / 256) * double(rows / 64 + 1);  // 64 rows per tile at least
    return;
  }
  p->places = 0;
  const int64_t rb = 8 * scalar_rt(d, rows);
  const int64_t ctas = (n + kRowsKeys - 1) / kRowsKeys * hkv, blocks = (rows + rb - 1) / rb;
  int64_t s = (kWeightsCtas + ctas - 1) / ctas;  // a few CTAs per SM
  if (s > blocks) s = blocks;
  if (s > 64) s = 64;
  p->rows_per_split = (blocks + s - 1) / s * rb;
  p->rsplit = int((rows + p->rows_per_split - 1) / p->rows_per_split);
  p->sum_floats = p->rsplit > 1 ? uint64_t(p->rsplit) * hkv * uint64_t(n) : 0;
}

// Floats of column sums that cover every call with at most n tokens: the splits of n' <= n tokens take
// ceil(kWeightsCtas / ctas) * hkv * n' <= 64 * kWeightsCtas + hkv * n floats.
uint64_t weights_sums_bound(int dtype, int hkv, int64_t n) {
  return (dtype == ZHA_BF16 ? weights_tc_floats() : uint64_t(kWeightsCtas) * kRowsKeys) + uint64_t(hkv) * uint64_t(n);
}

cudaError_t launch_weights(const WeightsArgs& a, int dtype, int d, cudaStream_t st) {
  if (a.logits) {
    count_launches(1);
    return launch_after(weights_logits_kernel, dim3(unsigned((a.n + 1023) / 1024), unsigned(a.hkv)), 256, 0, st, a);
  }
  if (dtype == ZHA_BF16) {
    if (a.acc_in != a.acc_out) return launch_weights_tc(a, d, st);
    // in place: the kernels add up behind the partial sums, and nothing of the caller's changes before all have ended
    WeightsArgs b = a;
    b.acc_out = a.sums + weights_tc_floats();
    b.ld_acc_out = a.n;
    const cudaError_t e = launch_weights_tc(b, d, st);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return launch_after(weights_commit_kernel, dim3(unsigned((a.n + 1023) / 1024), unsigned(a.hkv)), 256, 0, st, b, a.acc_out,
                        a.ld_acc_out);
  }
  count_launches(a.rsplit > 1 ? 2 : 1);
  const cudaError_t e = d == 128 ? run_weights_rt<float, 128>(a, st) : run_weights_rt<float, 64>(a, st);
  if (e != cudaSuccess || a.rsplit <= 1) return e;
  return launch_after(weights_join_kernel, dim3(unsigned((a.n + 255) / 256), unsigned(a.hkv)), 256, 0, st, a);
}

}  // namespace zha
