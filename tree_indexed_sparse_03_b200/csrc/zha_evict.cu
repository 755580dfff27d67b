// Eviction from a KV cache by accumulated attention weight (zha_cache_evict):
// per KV head the tokens to keep, then the kept rows of K, V and the sums
// moved to the front in token order.
#include <cooperative_groups.h>

#include "zha_rows.cuh"

namespace cg = cooperative_groups;

namespace zha {

// ------------------------------------------------------------------ selection
// The keep - first - last largest sums among tokens [first, n - last), ties to
// the lower token.  One cluster of 8 CTAs per KV head, each with a contiguous
// eighth of the tokens.  The threshold is found most significant bits first, 11 +
// 11 + 10 bits: shared-memory histograms, added over the cluster through distributed
// shared memory (every CTA reads all eight, so no second exchange is needed).
// Then each warp counts the tokens above and at the threshold in its own run of tokens, one scan over
// warps and CTAs gives its output position, and it lists its kept tokens in order.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCtas = 8;  // the portable cluster size
constexpr int kSelBins = 2048;

// Larger sum, larger key; NaN below everything; -0 equal to +0.
__device__ __forceinline__ uint32_t evict_key(float x) {
  if (x != x) return 0u;
  return float_to_ordered(x == 0.f ? 0.f : x);
}

__global__ void __cluster_dims__(kSelCtas, 1, 1) __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ uint32_t hist[kSelBins];
  __shared__ uint32_t wsum[kSelWarps];
  __shared__ uint32_t found[2];                // bin of the threshold, tokens above it
  __shared__ uint32_t wgt[kSelWarps], weq[kSelWarps];
  __shared__ uint32_t cta_cnt[2];              // tokens above / at the threshold of this CTA
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, rank = int(cl.block_rank());
  const int h = blockIdx.x / kSelCtas;
  const float* acc = a.acc + int64_t(h) * a.ld_acc;
  int32_t* out = a.idx + int64_t(h) * a.keep;
  for (int64_t i = int64_t(rank) * kSelThreads + tid; i < a.first + a.last; i += int64_t(kSelCtas) * kSelThreads) {
    if (i < a.first) out[i] = int32_t(i);
    else out[a.keep - a.last + (i - a.first)] = int32_t(a.n - a.last + (i - a.first));
  }
  const int64_t n_mid = a.n - a.first - a.last;
  uint32_t want = uint32_t(a.keep - a.first - a.last);  // tokens still to take at or below the current prefix
  if (want == 0) return;  // the same for every CTA of the cluster
  // a warp's run of tokens, a multiple of 32 so that its rows are whole warp iterations
  const int64_t per = (n_mid + int64_t(kSelCtas) * kSelWarps * 32 - 1) / (int64_t(kSelCtas) * kSelWarps * 32) * 32;
  const int64_t t0 = min64(n_mid, (int64_t(rank) * kSelWarps + wid) * per);
  const int64_t t1 = min64(n_mid, t0 + per);
  const float* mid = acc + a.first;
  uint32_t prefix = 0, mask = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t bins = pass == 2 ? 1024u : 2048u;
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0u;
    __syncthreads();
    for (int64_t i = t0 + lane; i < t1; i += 32) {
      const uint32_t k = evict_key(__ldcg(mid + i));
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
    }
    cl.sync();
    // bins in descending order: thread t holds bins 2t and 2t + 1 from the top
    uint32_t v[2] = {0u, 0u};
#pragma unroll
    for (int q = 0; q < kSelCtas; ++q) {
      const uint32_t* r = cl.map_shared_rank(hist, q);
      v[0] += r[kSelBins - 1 - 2 * tid];
      v[1] += r[kSelBins - 2 - 2 * tid];
    }
    uint32_t inc = v[0] + v[1];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += y;
    }
    if (lane == 31) wsum[wid] = inc;
    __syncthreads();
    uint32_t before = 0;
    {
      uint32_t w = wsum[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += y;
      }
      const uint32_t up = __shfl_sync(0xffffffffu, w, (wid + 31) & 31);
      before = wid == 0 ? 0u : up;
    }
    before += inc - v[0] - v[1];
    if (before < want && before + v[0] >= want) {
      found[0] = uint32_t(kSelBins - 1 - 2 * tid);
      found[1] = before;
    } else if (before + v[0] < want && before + v[0] + v[1] >= want) {
      found[0] = uint32_t(kSelBins - 2 - 2 * tid);
      found[1] = before + v[0];
    }
    cl.sync();  // every CTA has read the histograms; `found` is visible to this CTA
    prefix |= found[0] << shift;
    mask |= (bins - 1) << shift;
    want -= found[1];
    __syncthreads();
  }
  // prefix is the threshold key; `want` of the tokens at it are kept, the lowest ones
  uint32_t gt = 0, eq = 0;
  for (int64_t i = t0 + lane; i < t1; i += 32) {
    const uint32_t k = evict_key(__ldcg(mid + i));
    gt += k > prefix;
    eq += k == prefix;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, off);
    eq += __shfl_xor_sync(0xffffffffu, eq, off);
  }
  if (lane == 0) {
    wgt[wid] = gt;
    weq[wid] = eq;
  }
  __syncthreads();
  uint32_t g = wgt[lane], e = weq[lane], gsum = g, esum = e;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    gsum += __shfl_xor_sync(0xffffffffu, gsum, off);
    esum += __shfl_xor_sync(0xffffffffu, esum, off);
  }
  if (tid == 0) {
    cta_cnt[0] = gsum;
    cta_cnt[1] = esum;
  }
  uint32_t gpre = lane < wid ? g : 0u, epre = lane < wid ? e : 0u;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    gpre += __shfl_xor_sync(0xffffffffu, gpre, off);
    epre += __shfl_xor_sync(0xffffffffu, epre, off);
  }
  cl.sync();
  for (int q = 0; q < rank; ++q) {
    const uint32_t* r = cl.map_shared_rank(cta_cnt, q);
    gpre += r[0];
    epre += r[1];
  }
  for (int64_t i0 = t0; i0 < t1; i0 += 32) {
    const int64_t i = i0 + lane;
    const bool in = i < t1;
    const uint32_t k = in ? evict_key(__ldcg(mid + i)) : 0u;
    const bool is_gt = in && k > prefix, is_eq = in && k == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t ge = gpre + __popc(bg & below), ee = epre + __popc(be & below);
    if (is_gt || (is_eq && ee < want)) out[a.first + ge + (ee < want ? ee : want)] = int32_t(a.first + i);
    gpre += __popc(bg);
    epre += __popc(be);
  }
  cl.sync();  // no CTA leaves while another reads its shared memory
}

// ------------------------------------------------------------------ moving the rows
// Separate outputs: a plain gather.  Each thread moves four 16-byte pieces, kMoveRows kept
// rows apart, so that four loads are in flight; bound by HBM (each kept row read and
// written once).
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

__global__ void __launch_bounds__(kMoveThreads) evict_gather_kernel(EvictArgs a) {
  const int h = blockIdx.y;
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
  evict_select_kernel<<<unsigned(a.hkv) * kSelCtas, kSelThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.in_place) {
    evict_slide_kernel<<<dim3(unsigned(a.row_bytes / 32 * 2 + 1), unsigned(a.hkv)), kSlideThreads, 0, st>>>(a);
  } else {
    const int64_t pieces = a.keep * (a.row_bytes / 16);
    const unsigned gx = unsigned((pieces + kMoveThreads * kMoveUnroll - 1) / (kMoveThreads * kMoveUnroll));
    evict_gather_kernel<<<dim3(gx, unsigned(a.hkv), 3), kMoveThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace zha
