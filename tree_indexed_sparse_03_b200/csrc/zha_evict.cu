// Eviction from a KV cache by accumulated attention weight (zha_cache_evict):
// per KV head the tokens to keep, then the kept rows of K, V and the sums
// moved to the front in token order.
#include "zha_rows.cuh"

namespace zha {

// ------------------------------------------------------------------ selection
// The keep - first - last largest sums among tokens [first, n - last), ties to the lower token.  The threshold is
// found most significant bits first, 11 + 11 + 10 bits, from histograms of the ordered keys; then each warp counts
// the tokens above and at the threshold in its run of tokens, a scan gives its output position, and it lists its
// kept tokens in order.  What bounds it is latency: up to 16K tokens one CTA per head keeps all keys in registers
// (4K tokens 5 us; read again from L2 in each pass 25 us), above that the passes are kernels over the whole GPU (a
// cluster of eight CTAs per head took 34 us for 256K tokens and 142 us for 1M, with four heads; these 18 and 50).
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;

// Larger sum, larger key; NaN below everything; -0 equal to +0.
__device__ __forceinline__ uint32_t evict_key(float x) {
  if (x != x) return 0u;
  return float_to_ordered(x == 0.f ? 0.f : x);
}

// The bin that holds the want-th largest key and the keys above that bin, from a histogram of kSelBins bins (thread
// t holds bins 2t and 2t + 1 from the top); the result is in found[] after the next barrier.
__device__ __forceinline__ void sel_find(const uint32_t* hist, uint32_t want, uint32_t* wsum, uint32_t* found) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const uint2 two = *reinterpret_cast<const uint2*>(hist + kSelBins - 2 - 2 * tid);
  const uint32_t v[2] = {two.y, two.x};
  uint32_t inc = v[0] + v[1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += y;
  }
  if (lane == 31) wsum[wid] = inc;
  __syncthreads();
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < wid ? wsum[lane] : 0u) + inc - v[0] - v[1];
  if (before < want && before + v[0] >= want) {
    found[0] = uint32_t(kSelBins - 1 - 2 * tid);
    found[1] = before;
  } else if (before + v[0] < want && before + v[0] + v[1] >= want) {
    found[0] = uint32_t(kSelBins - 2 - 2 * tid);
    found[1] = before + v[0];
  }
}

__device__ __forceinline__ int sel_shift(int pass) { return pass == 0 ? 21 : (pass == 1 ? 10 : 0); }
__device__ __forceinline__ uint32_t sel_mask(int pass) { return pass == 2 ? 1023u : 2047u; }

// A thread's keys: RK rounds of 32 tokens of its warp's run [t0, t1).
template <int RK>
__device__ __forceinline__ void sel_load(const float* mid, int t0, int t1, uint32_t* keys) {
  const int lane = threadIdx.x & 31;
  float v[RK];
#pragma unroll
  for (int j = 0; j < RK; ++j) {
    const int i = t0 + 32 * j + lane;
    v[j] = i < t1 ? __ldcg(mid + i) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < RK; ++j) keys[j] = evict_key(v[j]);
}

template <int RK>
__device__ __forceinline__ void sel_count(const uint32_t* keys, int t0, int t1, uint32_t prefix, uint32_t* gt, uint32_t* eq) {
  const int lane = threadIdx.x & 31;
  uint32_t g = 0, e = 0;
#pragma unroll
  for (int j = 0; j < RK; ++j) {
    const bool live = t0 + 32 * j + lane < t1;
    g += live && keys[j] > prefix;
    e += live && keys[j] == prefix;
  }
  *gt = __reduce_add_sync(0xffffffffu, g);
  *eq = __reduce_add_sync(0xffffffffu, e);
}

// A warp lists its kept tokens: gpre keys above the threshold and epre at it come before its run.
template <int RK>
__device__ __forceinline__ void sel_list(const uint32_t* keys, int t0, int t1, uint32_t prefix, uint32_t want, uint32_t gpre,
                                         uint32_t epre, int first, int32_t* out) {
  const int lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int j = 0; j < RK; ++j) {
    const int i = t0 + 32 * j + lane;
    const bool live = i < t1, is_gt = live && keys[j] > prefix, is_eq = live && keys[j] == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const uint32_t ge = gpre + __popc(bg & below), ee = epre + __popc(be & below);
    if (is_gt || (is_eq && ee < want)) out[first + ge + (ee < want ? ee : want)] = first + i;
    gpre += __popc(bg);
    epre += __popc(be);
  }
}

// The tokens kept whatever their sums, by `threads` threads.
__device__ __forceinline__ void sel_ends(const EvictArgs& a, int32_t* out, int64_t thread, int64_t threads) {
  for (int64_t i = thread; i < a.first + a.last; i += threads) {
    if (i < a.first) out[i] = int32_t(i);
    else out[a.keep - a.last + (i - a.first)] = int32_t(a.n - a.last + (i - a.first));
  }
}

// Short caches: one CTA per head, all keys in its registers.
template <int RK> __global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  __shared__ __align__(8) uint32_t hist[kSelBins];
  __shared__ uint32_t wsum[kSelWarps], found[2], wgt[kSelWarps], weq[kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, h = blockIdx.x;
  int32_t* out = a.idx + int64_t(h) * a.keep;
  pdl_trigger();
  pdl_wait();
  sel_ends(a, out, tid, kSelThreads);
  const int n_mid = int(a.n - a.first - a.last);
  uint32_t want = uint32_t(a.keep - a.first - a.last);  // tokens still to take at or below the current prefix
  if (want == 0) return;
  // a warp's run of tokens, a multiple of 32 so that its rounds are whole
  const int per = (n_mid + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
  const int t0 = min(n_mid, wid * per), t1 = min(n_mid, t0 + per);
  uint32_t keys[RK];
  sel_load<RK>(a.acc + int64_t(h) * a.ld_acc + a.first, t0, t1, keys);
  uint32_t prefix = 0, mask = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = sel_shift(pass);
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0u;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < RK; ++j)
      if (t0 + 32 * j + lane < t1 && (keys[j] & mask) == prefix) atomicAdd(&hist[(keys[j] >> shift) & sel_mask(pass)], 1u);
    __syncthreads();
    sel_find(hist, want, wsum, found);
    __syncthreads();
    prefix |= found[0] << shift;
    mask |= sel_mask(pass) << shift;
    want -= found[1];
  }
  // prefix is the threshold key; `want` of the tokens at it are kept, the lowest ones
  uint32_t gt, eq;
  sel_count<RK>(keys, t0, t1, prefix, &gt, &eq);
  if (lane == 0) {
    wgt[wid] = gt;
    weq[wid] = eq;
  }
  __syncthreads();
  sel_list<RK>(keys, t0, t1, prefix, want, __reduce_add_sync(0xffffffffu, lane < wid ? wgt[lane] : 0u),
               __reduce_add_sync(0xffffffffu, lane < wid ? weq[lane] : 0u), int(a.first), out);
}

// Long caches: chunks of 8192 tokens over the whole GPU, one kernel per pass; the histograms are added in global
// memory (an integer sum, the same in any order).  Kernel `pass` = 0, 1, 2 adds the pass's histogram, 3 counts each
// chunk's keys above and at the threshold, 4 lists.  Every kernel finds the bin of the pass before it from that
// histogram (all CTAs the same one; the first leaves it for the kernels after the next).
constexpr int kWideKeys = 8;
constexpr int kWideChunk = kSelThreads * kWideKeys;

struct WideState {       // of one head
  uint32_t hist[3][kSelBins];
  uint32_t prefix[4], want[4];  // after pass 0, 1, 2 (entries 1..3)
};

__global__ void __launch_bounds__(kSelThreads) evict_wide_kernel(EvictArgs a, int pass, int chunks) {
  __shared__ __align__(8) uint32_t hist[kSelBins];
  __shared__ uint32_t wsum[kSelWarps], found[2], wgt[kSelWarps], weq[kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, h = blockIdx.y;
  WideState* s = reinterpret_cast<WideState*>(a.scratch) + h;
  uint32_t* counts = reinterpret_cast<uint32_t*>(reinterpret_cast<WideState*>(a.scratch) + a.hkv) + int64_t(h) * chunks * 2;
  const int n_mid = int(a.n - a.first - a.last);
  const float* mid = a.acc + int64_t(h) * a.ld_acc + a.first;
  int32_t* out = a.idx + int64_t(h) * a.keep;
  // the histogram passes take every gridDim.x-th chunk, the others have one CTA per chunk
  int chunk = blockIdx.x;
  int t0 = min(n_mid, chunk * kWideChunk + wid * kWideKeys * 32), t1 = min(n_mid, t0 + kWideKeys * 32);
  uint32_t keys[kWideKeys];
  sel_load<kWideKeys>(mid, t0, t1, keys);
  pdl_trigger();
  if (pass == 0) sel_ends(a, out, int64_t(blockIdx.x) * kSelThreads + tid, int64_t(gridDim.x) * kSelThreads);
  else pdl_wait();
  uint32_t prefix = 0, mask = 0, want = uint32_t(a.keep - a.first - a.last);
  if (pass > 1) {
    prefix = __ldcg(&s->prefix[pass - 1]);
    want = __ldcg(&s->want[pass - 1]);
  }
  if (pass > 0 && pass < 4) {
    const int done = pass - 1;  // the pass whose histogram is complete
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = __ldcg(&s->hist[done][i]);
    __syncthreads();
    sel_find(hist, want, wsum, found);
    __syncthreads();
    prefix |= found[0] << sel_shift(done);
    want -= found[1];
    if (blockIdx.x == 0 && tid == 0) {
      s->prefix[pass] = prefix;
      s->want[pass] = want;
    }
    mask = ~((1u << sel_shift(done)) - 1u);
  }
  if (pass < 3) {
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0u;
    __syncthreads();
    while (true) {
#pragma unroll
      for (int j = 0; j < kWideKeys; ++j)
        if (t0 + 32 * j + lane < t1 && (keys[j] & mask) == prefix)
          atomicAdd(&hist[(keys[j] >> sel_shift(pass)) & sel_mask(pass)], 1u);
      chunk += gridDim.x;
      if (chunk >= chunks) break;
      t0 = min(n_mid, chunk * kWideChunk + wid * kWideKeys * 32);
      t1 = min(n_mid, t0 + kWideKeys * 32);
      sel_load<kWideKeys>(mid, t0, t1, keys);
    }
    __syncthreads();
    for (int i = tid; i < kSelBins; i += kSelThreads)
      if (hist[i]) atomicAdd(&s->hist[pass][i], hist[i]);
    return;
  }
  uint32_t gt, eq;
  sel_count<kWideKeys>(keys, t0, t1, prefix, &gt, &eq);
  if (lane == 0) {
    wgt[wid] = gt;
    weq[wid] = eq;
  }
  __syncthreads();
  if (pass == 3) {
    if (wid == 0) {
      gt = __reduce_add_sync(0xffffffffu, wgt[lane]);
      eq = __reduce_add_sync(0xffffffffu, weq[lane]);
      if (lane == 0) {
        counts[2 * chunk] = gt;
        counts[2 * chunk + 1] = eq;
      }
    }
    return;
  }
  uint32_t gpre = lane < wid ? wgt[lane] : 0u, epre = lane < wid ? weq[lane] : 0u;
  for (int q = lane; q < chunk; q += 32) {
    gpre += __ldcg(counts + 2 * q);
    epre += __ldcg(counts + 2 * q + 1);
  }
  sel_list<kWideKeys>(keys, t0, t1, prefix, want, __reduce_add_sync(0xffffffffu, gpre), __reduce_add_sync(0xffffffffu, epre),
                      int(a.first), out);
}

constexpr int kShortMost = 16 * kSelThreads;  // up to here one CTA holds all keys (30K tokens: 22 us with 32 a thread, 16 us over
                                              // the whole GPU)

static int64_t wide_chunks(int64_t mid) { return (mid + kWideChunk - 1) / kWideChunk; }

// Scratch of the long caches' selection over n tokens (whatever first and last are).
uint64_t evict_scratch_bytes(int hkv, int64_t n) {
  return n <= kShortMost ? 0 : uint64_t(hkv) * (sizeof(WideState) + uint64_t(wide_chunks(n)) * 8);
}

template <int RK> static cudaError_t run_select(const EvictArgs& a, cudaStream_t st) {
  count_launches(1);
  return launch_after(evict_select_kernel<RK>, dim3(unsigned(a.hkv)), kSelThreads, 0, st, a);
}

static cudaError_t launch_select(const EvictArgs& a, cudaStream_t st) {
  const int64_t mid = a.n - a.first - a.last;
  if (mid <= 4 * kSelThreads || a.keep == a.first + a.last) return run_select<4>(a, st);
  if (mid <= kShortMost) return run_select<16>(a, st);
  count_launches(5);
  cudaError_t e = cudaMemsetAsync(a.scratch, 0, size_t(a.hkv) * sizeof(WideState), st);
  if (e != cudaSuccess) return e;
  const int chunks = int(wide_chunks(mid));
  const int few = int(min64(chunks, (2 * 148 + a.hkv - 1) / a.hkv));  // two CTAs per SM: one merge into the global histogram each
  evict_wide_kernel<<<dim3(unsigned(few), unsigned(a.hkv)), kSelThreads, 0, st>>>(a, 0, chunks);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  for (int pass = 1; pass < 5; ++pass) {
    const dim3 grid(unsigned(pass < 3 ? few : chunks), unsigned(a.hkv));
    if ((e = launch_after(evict_wide_kernel, grid, kSelThreads, 0, st, a, pass, chunks)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// ------------------------------------------------------------------ moving the rows
// Separate outputs: a plain gather.  Each thread has four 16-byte pieces in flight; bound by HBM (each kept row read
// and written once).  1M -> 512K tokens, 4 heads of 128 bf16: 443 us with the selection.  In the run that compared them
// 128 threads and streaming stores took 435, 256 and plain stores 465, eight pieces 507, two 489.
constexpr int kMoveThreads = 128;
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
    if (i < pieces) __stcs(reinterpret_cast<uint4*>(dst + i * 16), v[u]);  // not read again soon
  }
}

// Outputs that are their own inputs: kept row j comes from idx[j] >= j, so rows must be read before an
// earlier-listed row's place is written.  One CTA moves a 32-byte column slice of one head's K or V (or its sums):
// rounds of kSlideRows rows, all of a round's loads before a barrier, its stores after it.  Writing rows [i, i +
// kSlideRows) can only overwrite sources of rows before i + kSlideRows, which have all been read; slices share no
// bytes, so CTAs need no order among themselves.  Bound by latency: a CTA has one round of loads in flight and few
// CTAs share the work (4 heads of 128 bf16: 68, one head of 64 bf16: 9).  With the selection 256K -> 64K tokens take 156
// us and 1M -> 512K 1,092 us for 4 heads of 128 bf16 (other buffers: 74 and 451), 256K -> 64K 140 us for one head of 64
// (32).
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
  count_launches(1);
  const cudaError_t e = launch_select(a, st);
  if (e != cudaSuccess) return e;
  if (a.in_place)
    return launch_after(evict_slide_kernel, dim3(unsigned(a.row_bytes / 32 * 2 + 1), unsigned(a.hkv)), kSlideThreads, 0, st, a);
  const int64_t pieces = a.keep * (a.row_bytes / 16);
  const unsigned gx = unsigned((pieces + kMoveThreads * kMoveUnroll - 1) / (kMoveThreads * kMoveUnroll));
  return launch_after(evict_gather_kernel, dim3(gx, unsigned(a.hkv), 3), kMoveThreads, 0, st, a);
}

}  // namespace zha
