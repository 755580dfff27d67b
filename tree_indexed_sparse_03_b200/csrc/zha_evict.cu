// Eviction from a KV cache by accumulated attention weight (zha_cache_evict):
// per KV head the tokens to keep, then the kept rows of K, V and the sums
// moved to the front in token order.
#include <cooperative_groups.h>

#include "zha_rows.cuh"

namespace cg = cooperative_groups;

namespace zha {

// ------------------------------------------------------------------ selection
// The keep - first - last largest sums among tokens [first, n - last), ties to
// the lower token.  CTAS CTAs per KV head (one, or a cluster), each warp with a contiguous run of tokens.
// The threshold is found most significant bits first, 11 + 11 + 10 bits: shared-memory histograms, added over the
// cluster through distributed shared memory (every CTA reads all of them, so no second
// exchange is needed).  Then each warp counts the tokens above and at the threshold in its run, one scan over warps
// and CTAs gives its output position, and it lists its kept tokens in order.
// The sums are read once: RK of them stay in each thread's registers as ordered keys (RK = 0: too many,
// read again in each of the five passes, from L2).  What is left is latency: each pass ends in two
// barriers and a scan.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelCluster = 8;  // the portable cluster size

// Larger sum, larger key; NaN below everything; -0 equal to +0.
__device__ __forceinline__ uint32_t evict_key(float x) {
  if (x != x) return 0u;
  return float_to_ordered(x == 0.f ? 0.f : x);
}

template <int CTAS> __device__ __forceinline__ void sel_sync() {
  if (CTAS > 1) cg::this_cluster().sync();
  else __syncthreads();
}

// f(key, live) for each 32 tokens of a warp's run [t0, t1) in order; live: the lane has a token.
template <int RK, typename F>
__device__ __forceinline__ void sel_each(const uint32_t* regs, const float* mid, int t0, int t1, F f) {
  const int lane = threadIdx.x & 31;
  if (RK > 0) {
#pragma unroll
    for (int j = 0; j < RK; ++j) f(regs[j], t0 + 32 * j + lane < t1, t0 + 32 * j + lane);
  } else {
    for (int i0 = t0; i0 < t1; i0 += 256) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + 32 * j + lane;
        v[j] = i < t1 ? __ldcg(mid + i) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f(evict_key(v[j]), i0 + 32 * j + lane < t1, i0 + 32 * j + lane);
    }
  }
}

template <int CTAS, int RK> __global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  __shared__ uint32_t hist[kSelBins];
  __shared__ uint32_t wsum[kSelWarps];
  __shared__ uint32_t found[2];  // bin of the threshold, tokens above it
  __shared__ uint32_t wgt[kSelWarps], weq[kSelWarps];
  __shared__ uint32_t cta_cnt[2];  // tokens above / at the threshold of this CTA
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = CTAS > 1 ? int(cg::this_cluster().block_rank()) : 0;
  const int h = blockIdx.x / CTAS;
  int32_t* out = a.idx + int64_t(h) * a.keep;
  pdl_trigger();
  for (int64_t i = int64_t(rank) * kSelThreads + tid; i < a.first + a.last; i += int64_t(CTAS) * kSelThreads) {
    if (i < a.first) out[i] = int32_t(i);
    else out[a.keep - a.last + (i - a.first)] = int32_t(a.n - a.last + (i - a.first));
  }
  const int n_mid = int(a.n - a.first - a.last);
  uint32_t want = uint32_t(a.keep - a.first - a.last);  // tokens still to take at or below the current prefix
  if (want == 0) return;  // the same for every CTA of the cluster
  // a warp's run of tokens, a multiple of 32 so that its rows are whole warp iterations
  const int64_t per = (int64_t(n_mid) + CTAS * kSelWarps * 32 - 1) / (CTAS * kSelWarps * 32) * 32;
  const int t0 = int(min64(n_mid, (int64_t(rank) * kSelWarps + wid) * per)), t1 = int(min64(n_mid, t0 + per));
  const float* mid = a.acc + int64_t(h) * a.ld_acc + a.first;
  uint32_t keys[RK > 0 ? RK : 1];
  if (RK > 0) {
    float v[RK > 0 ? RK : 1];
#pragma unroll
    for (int j = 0; j < RK; ++j) {
      const int i = t0 + 32 * j + lane;
      v[j] = i < t1 ? __ldcg(mid + i) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < RK; ++j) keys[j] = evict_key(v[j]);
  }
  uint32_t prefix = 0, mask = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t bins = pass == 2 ? 1024u : 2048u;
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0u;
    __syncthreads();
    sel_each<RK>(keys, mid, t0, t1, [&](uint32_t k, bool live, int) {
      if (live && (k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
    });
    sel_sync<CTAS>();
    // bins in descending order: thread t holds bins 2t and 2t + 1 from the top
    uint32_t v[2] = {0u, 0u};
#pragma unroll
    for (int q = 0; q < CTAS; ++q) {
      const uint32_t* r = CTAS > 1 ? cg::this_cluster().map_shared_rank(hist, q) : hist;
      const uint2 two = *reinterpret_cast<const uint2*>(r + kSelBins - 2 - 2 * tid);
      v[0] += two.y;
      v[1] += two.x;
    }
    uint32_t inc = v[0] + v[1];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += y;
    }
    if (lane == 31) wsum[wid] = inc;
    __syncthreads();
    uint32_t before = __reduce_add_sync(0xffffffffu, lane < wid ? wsum[lane] : 0u) + inc - v[0] - v[1];
    if (before < want && before + v[0] >= want) {
      found[0] = uint32_t(kSelBins - 1 - 2 * tid);
      found[1] = before;
    } else if (before + v[0] < want && before + v[0] + v[1] >= want) {
      found[0] = uint32_t(kSelBins - 2 - 2 * tid);
      found[1] = before + v[0];
    }
    sel_sync<CTAS>();  // every CTA has read the histograms; `found` is visible to this CTA
    prefix |= found[0] << shift;
    mask |= (bins - 1) << shift;
    want -= found[1];
  }
  // prefix is the threshold key; `want` of the tokens at it are kept, the lowest ones
  uint32_t gt = 0, eq = 0;
  sel_each<RK>(keys, mid, t0, t1, [&](uint32_t k, bool live, int) {
    gt += live && k > prefix;
    eq += live && k == prefix;
  });
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    wgt[wid] = gt;
    weq[wid] = eq;
  }
  __syncthreads();
  uint32_t gpre = __reduce_add_sync(0xffffffffu, lane < wid ? wgt[lane] : 0u);
  uint32_t epre = __reduce_add_sync(0xffffffffu, lane < wid ? weq[lane] : 0u);
  if (CTAS > 1) {
    if (tid == kSelThreads - 1) {
      cta_cnt[0] = gpre + gt;
      cta_cnt[1] = epre + eq;
    }
    sel_sync<CTAS>();
    for (int q = 0; q < rank; ++q) {
      const uint32_t* r = cg::this_cluster().map_shared_rank(cta_cnt, q);
      gpre += r[0];
      epre += r[1];
    }
  }
  sel_each<RK>(keys, mid, t0, t1, [&](uint32_t k, bool live, int i) {
    const bool is_gt = live && k > prefix, is_eq = live && k == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t ge = gpre + __popc(bg & below), ee = epre + __popc(be & below);
    if (is_gt || (is_eq && ee < want)) out[a.first + ge + (ee < want ? ee : want)] = int32_t(a.first + i);
    gpre += __popc(bg);
    epre += __popc(be);
  });
  if (CTAS > 1) sel_sync<CTAS>();  // no CTA leaves while another reads its shared memory
}

template <int CTAS, int RK> cudaError_t run_select(const EvictArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(unsigned(a.hkv) * CTAS);
  c.blockDim = dim3(kSelThreads);
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CTAS;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = CTAS > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&c, evict_select_kernel<CTAS, RK>, a);
}

// One CTA where its registers hold all keys without waiting for a cluster; a cluster of eight above, its registers up to
// 256K tokens.
static cudaError_t launch_select(const EvictArgs& a, cudaStream_t st) {
  const int64_t mid = a.n - a.first - a.last;
  if (mid <= 4 * kSelThreads) return run_select<1, 4>(a, st);
  if (mid <= 16 * kSelThreads) return run_select<1, 16>(a, st);
  if (mid <= 8 * kSelThreads * kSelCluster) return run_select<kSelCluster, 8>(a, st);
  if (mid <= 32 * kSelThreads * kSelCluster) return run_select<kSelCluster, 32>(a, st);
  return run_select<kSelCluster, 0>(a, st);
}

// ------------------------------------------------------------------ moving the rows
// Separate outputs: a plain gather.  Each thread moves four 16-byte pieces, kMoveRows kept
// rows apart, so that four loads are in flight; bound by HBM (each kept row read and
// written once).
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

__global__ void __launch_bounds__(kMoveThreads) evict_gather_kernel(EvictArgs a) {
  const int h = blockIdx.y;
  pdl_wait();
  const int cpr = a.row_bytes / 16;  // 16-byte pieces per row: 8, 16 or 32
  const int64_t pieces = a.keep * cpr;
  const int32_t* idx = a.idx + int64_t(h) * a.keep;
  const int64_t i0 = int64_t(blockIdx.x) * kMoveThreads * kMoveUnroll + threadIdx.x;
  if (blockIdx.z == 2) {
    const float* src = a.acc + h * a.ld_acc;
    float* dst = a.acc_out + h * a.ld_acc_out;
    for (int64_t i = int64_t(blockIdx.x) * kMoveThreads + threadIdx.x; i < a.keep;
         i += int64_t(gridDim.x) * kMoveThreads)
      dst[i] = src[idx[i]];
    return;
  }
  const char* src = static_cast<const char*>(blockIdx.z ? a.V : a.K) + h * a.ld * a.row_bytes;
  char* dst = static_cast<char*>(blockIdx.z ? a.V_out : a.K_out) + h * a.ld_out * a.row_bytes;
  uint4 v[kMoveUnroll];
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    const int64_t i = i0 + u * kMoveThreads;
    if (i < pieces) v[u] = ldg_stream(src + int64_t(idx[i / cpr]) * a.row_bytes + (i % cpr) * 16);
  }
#pragma unroll
  for (int u = 0; u < kMoveUnroll; ++u) {
    const int64_t i = i0 + u * kMoveThreads;
    if (i < pieces) *reinterpret_cast<uint4*>(dst + i * 16) = v[u];
  }
}

// Outputs that are their own inputs: kept row j comes from idx[j] >= j, so rows must be read before an
// earlier-listed row's place is written.  One CTA moves a 32-byte column slice of one head's K or V (or its
// sums): rounds of kSlideRows rows, all of a round's loads before a barrier, its stores after it.  Writing rows [i, i +
// kSlideRows) can only overwrite sources of rows before i + kSlideRows, which have all been read; slices share no bytes,
// so CTAs need no order among themselves.
constexpr int kSlideThreads = 1024;
constexpr int kSlideUnroll = 4;

template <typename E> __device__ __forceinline__ void slide_rows(const char* src, char* dst, const int32_t* idx,
                                                                 int64_t keep, int64_t stride, int lanes) {
  const int per = kSlideThreads / lanes * kSlideUnroll;  // rows of a round
  const int sub = threadIdx.x % lanes, r = threadIdx.x / lanes, step = kSlideThreads / lanes;
  for (int64_t j0 = 0; j0 < keep; j0 += per) {
    E v[kSlideUnroll];
#pragma unroll
    for (int u = 0; u < kSlideUnroll; ++u) {
      const int64_t j = j0 + r + u * step;
      if (j < keep) v[u] = __ldcg(reinterpret_cast<const E*>(src + int64_t(idx[j]) * stride) + sub);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSlideUnroll; ++u) {
      const int64_t j = j0 + r + u * step;
      if (j < keep) __stcg(reinterpret_cast<E*>(dst + j * stride) + sub, v[u]);
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kSlideThreads) evict_slide_kernel(EvictArgs a) {
  const int h = blockIdx.y, slices = a.row_bytes / 32;
  const int32_t* idx = a.idx + int64_t(h) * a.keep;
  const int x = blockIdx.x;
  pdl_wait();
  if (x < 2 * slices) {
    const bool v = x >= slices;
    const int64_t off = int64_t(x - (v ? slices : 0)) * 32;
    slide_rows<uint4>(static_cast<const char*>(v ? a.V : a.K) + h * a.ld * a.row_bytes + off,
                      static_cast<char*>(v ? a.V_out : a.K_out) + h * a.ld_out * a.row_bytes + off, idx, a.keep,
                      a.row_bytes, 2);
    return;
  }
  slide_rows<float>(reinterpret_cast<const char*>(a.acc + h * a.ld_acc),
                    reinterpret_cast<char*>(a.acc_out + h * a.ld_acc_out), idx, a.keep, 4, 1);
  if (a.acc_out == a.acc)  // the places that fall free belong to tokens still to come
    for (int64_t i = a.keep + threadIdx.x; i < a.n; i += kSlideThreads) a.acc_out[h * a.ld_acc_out + i] = 0.f;
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  count_launches(2);
  const cudaError_t e = launch_select(a, st);
  if (e != cudaSuccess) return e;
  if (a.in_place)
    return launch_after(evict_slide_kernel, dim3(unsigned(a.row_bytes / 32 * 2 + 1), unsigned(a.hkv)), kSlideThreads, 0, st, a);
  const int64_t pieces = a.keep * (a.row_bytes / 16);
  const unsigned gx = unsigned((pieces + kMoveThreads * kMoveUnroll - 1) / (kMoveThreads * kMoveUnroll));
  return launch_after(evict_gather_kernel, dim3(gx, unsigned(a.hkv), 3), kMoveThreads, 0, st, a);
}

}  // namespace zha
