// Arguments and work split shared by the kernels that attend many query rows
// over one KV cache: zha_prefix_decode and zha_dense_weights.
//
// Rows.  One KV head serves `group` query heads; the rows of KV head h are the
// (sequence b, query token i, head g) triples in that order, row index
// (b * m + i) * group + g.  The shared tokens [0, n) are attended by all rows of
// the head (row block = up to `rb` rows), a sequence's own tokens by its m * group
// rows.
//
// Work split.  A segment is one row block over one key range: first the
// prefix segments (h, row block), then the own segments (b, h, row block of the
// sequence).  A segment is cut into key tiles; the tiles of all segments, each
// segment followed by `extra` empty places for what starting one costs, form one flat list, and the CTAs take equal
// contiguous shares of it (the first T % nc one place more), so every CTA has the same work whatever
// the lengths are, lengths that only the device knows included.  A CTA leaves one partial (running max, running
// sum, numerator) per segment it shares with others; rows_combine_kernel joins them in CTA order.
#pragma once

#include <atomic>

#include "zha_args.cuh"

namespace zha {

struct RowsArgs {
  const void* K;            // [hkv][ld][d], tokens [0, n) are read
  const void* V;            // NULL: no outputs, only the rows' log-sum-exp
  const void* Ko;           // own caches [B][hkv][ld_own][d] (NULL: none)
  const void* Vo;
  const int32_t* own_len;   // [B] device
  const void* Q;            // [B][m][hq][d]
  float* O;                 // [B][m][hq][d] (NULL with V)
  float* lse;               // [B][m][hq] natural log, may be NULL
  float* part;              // partials: numerators, d floats per row
  float* part_tmp;          // tensor cores: [nc][rt] rows where the streams add up what they have so far
  float2* part_ml;          // and (running max in powers of two, running sum) per row
  float* logits;            // NULL, or [hkv][rows][ld_logits]: the prefix logits in powers of two (-inf where masked), kept
                            // for the weights pass
  int64_t ld_logits;
  int* status;
  int* plan;                // the flat list as the attention kernel's first CTA found it, for the join (rows_publish)
  int64_t ld, n, ld_own;
  int rows;                 // rows per KV head over the prefix: B * m * group
  int64_t part_own;         // first own slot's offset in `part`, in rows
  int B, m, hq, hkv, group;
  int causal;               // 1: query i sees prefix tokens [0, n - m + i] (B = 1)
  int has_own;
  int rb_log;               // rows per row block, a power of two
  int kt_log;               // keys per tile, a power of two
  int extra;                // empty places behind a segment's tiles
  int pp, po;               // row blocks of a prefix / an own segment
  int rp, ro;               // rows of a prefix / an own partial slot
  int rt;                   // rows of part_tmp per CTA
  int nc;                   // CTAs
  float scale;              // 1 / sqrt(d)
  long long wait_limit;     // bound of the waits on copies and products, SM cycles
};

// Tokens of sequence b's own cache (a length outside [0, ld_own] is clamped, so that no read leaves the cache).
__device__ __forceinline__ int64_t own_tokens(const RowsArgs& a, int b) {
  const int64_t v = a.own_len[b];
  return v < 0 ? 0 : min64(v, a.ld_own);
}

// Keys of the prefix that row r of a KV head sees (causal: its query token's position + 1).
__device__ __forceinline__ int64_t prefix_limit(const RowsArgs& a, int r) {
  return a.causal ? a.n - a.m + r / a.group + 1 : a.n;
}

// Own tokens that row r (within its sequence) sees: the m query tokens are the cache's last m.
__device__ __forceinline__ int64_t own_limit(const RowsArgs& a, int64_t len, int r) {
  const int64_t v = len - a.m + 1 + r / a.group;
  return v < 0 ? 0 : v;
}

// Tiles of the prefix segment of row block p (of every KV head).
__device__ __forceinline__ int prefix_tiles(const RowsArgs& a, int p) {
  const int last = min((p + 1) << a.rb_log, a.rows) - 1;
  return int((prefix_limit(a, last) + (1 << a.kt_log) - 1) >> a.kt_log);
}

__device__ __forceinline__ int own_tiles(const RowsArgs& a, int b) {
  return int((own_tokens(a, b) + (1 << a.kt_log) - 1) >> a.kt_log);
}

// Places of a segment of t tiles in the flat list.
__device__ __forceinline__ int seg_span(const RowsArgs& a, int t) { return t ? t + a.extra : 0; }

// Sum of f(i) over i in [0, n), by one full warp.
template <typename F> __device__ __forceinline__ int warp_total(int n, F f) {
  int s = 0;
  for (int i = threadIdx.x & 31; i < n; i += 32) s += f(i);
  return __reduce_add_sync(0xffffffffu, s);
}

// Contiguous shares of a list of `all` places for nc CTAs; the first `more` shares have one place more.  Where there
// are fewer places than CTAs the last CTAs have none.
struct Shares {
  int all, per, more;
  __device__ __forceinline__ void set(int total, int nc) {
    all = total;
    per = total / nc;
    more = total - per * nc;
  }
  __device__ __forceinline__ int begin(int c) const { return c * per + min(c, more); }
  __device__ __forceinline__ int owner(int x) const {
    const int big = more * (per + 1);
    return x < big ? x / (per + 1) : more + (x - big) / per;
  }
};

// The totals of the flat list, by one full warp.
struct RowsTotals {
  int head;    // places of one KV head's prefix segments
  int prefix;  // places of all prefix segments
  Shares sh;
};

__device__ __forceinline__ RowsTotals rows_totals(const RowsArgs& a) {
  RowsTotals t;
  t.head = a.causal ? warp_total(a.pp, [&](int p) { return seg_span(a, prefix_tiles(a, p)); })
                    : a.pp * seg_span(a, prefix_tiles(a, 0));
  t.prefix = t.head * a.hkv;
  t.sh.set(t.prefix + (a.has_own ? a.hkv * a.po * warp_total(a.B, [&](int b) { return seg_span(a, own_tiles(a, b)); }) : 0),
           a.nc);
  return t;
}

// First item of the list with lengths f(0..n) that holds position x (0 <= x < total), by one full warp; *base
// receives the position of the item's first element.
template <typename F> __device__ __forceinline__ int warp_find(int n, F f, int x, int* base) {
  const int lane = threadIdx.x & 31;
  int run = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int v = i0 + lane < n ? f(i0 + lane) : 0;
    int inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, run + inc > x);
    if (hit) {
      const int src = __ffs(hit) - 1;
      *base = __shfl_sync(0xffffffffu, run + inc - v, src);
      return i0 + src;
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  *base = run;
  return n;  // not reached for x < total
}

// A segment: its tiles are places [first, first + tiles) of the list, its empty places follow up to `next`.
struct RowsSeg {
  int own;        // 0: prefix, 1: own
  int b, h, p;    // sequence (own), KV head, row block
  int id;         // segment number
  int first, tiles, next;
};

// The segment that holds place x, by one full warp.
__device__ __forceinline__ RowsSeg rows_find(const RowsArgs& a, const RowsTotals& t, int x) {
  RowsSeg s;
  if (x < t.prefix) {
    s.own = 0;
    s.b = 0;
    s.h = x / t.head;
    const int r = x - s.h * t.head;
    int base;
    if (a.causal) {
      s.p = warp_find(a.pp, [&](int p) { return seg_span(a, prefix_tiles(a, p)); }, r, &base);
      s.tiles = prefix_tiles(a, s.p);
    } else {
      s.tiles = prefix_tiles(a, 0);
      s.p = r / seg_span(a, s.tiles);
      base = s.p * seg_span(a, s.tiles);
    }
    s.first = s.h * t.head + base;
    s.id = s.h * a.pp + s.p;
  } else {
    s.own = 1;
    const int per = a.hkv * a.po;
    int base;
    s.b = warp_find(a.B, [&](int b) { return seg_span(a, own_tiles(a, b)) * per; }, x - t.prefix, &base);
    s.tiles = own_tiles(a, s.b);
    const int u = (x - t.prefix - base) / seg_span(a, s.tiles);
    s.h = u / a.po;
    s.p = u - s.h * a.po;
    s.first = t.prefix + base + u * seg_span(a, s.tiles);
    s.id = a.hkv * a.pp + s.b * per + u;
  }
  s.next = s.first + seg_span(a, s.tiles);
  return s;
}

// Partial slot of CTA c for a segment.  With own caches every row has several partials: slot c + segment number
// (unique, since along the list either the CTA or the segment advances).  Without, a segment whose tiles lie inside
// one CTA's share is written out directly, and a share cuts at most two: slot 2c for one that holds the share's
// begin, 2c + 1 for a later one.  Returns the slot's first row in `part`.
__device__ __forceinline__ int64_t part_row(const RowsArgs& a, int c, int own, int id, bool later) {
  if (!a.has_own) return (2 * int64_t(c) + (later ? 1 : 0)) * a.rp;
  return own ? a.part_own + (int64_t(c) + id - a.hkv * a.pp) * a.ro : (int64_t(c) + id) * a.rp;
}

// Index of (sequence, query token, query head) of row r of KV head h in Q, O and lse (times d for Q and O).
__device__ __forceinline__ int64_t row_index(const RowsArgs& a, int h, int r) {
  const int t = r / a.group;
  return int64_t(t) * a.hq + h * a.group + (r - t * a.group);
}

// The list for the join, written once by one warp of the first CTA: places in all, of a head's prefix segments and of
// all of them; then the first place of every row block of a head and of every sequence's own segments (of one
// KV head and row block), both with their end.
__host__ __device__ __forceinline__ int64_t rows_plan_words(int pp, int B) { return 3 + pp + 1 + B + 1; }

template <typename F> __device__ __forceinline__ void warp_prefix(int n, F f, int* out) {
  const int lane = threadIdx.x & 31;
  int run = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int v = i0 + lane < n ? f(i0 + lane) : 0;
    int inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += y;
    }
    if (i0 + lane < n) out[i0 + lane] = run + inc - v;
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) out[n] = run;
}

__device__ __forceinline__ void rows_publish(const RowsArgs& a, const RowsTotals& t) {
  if ((threadIdx.x & 31) == 0) {
    a.plan[0] = t.sh.all;
    a.plan[1] = t.head;
    a.plan[2] = t.prefix;
  }
  warp_prefix(a.pp, [&](int p) { return seg_span(a, prefix_tiles(a, p)); }, a.plan + 3);
  if (a.has_own) warp_prefix(a.B, [&](int b) { return seg_span(a, own_tiles(a, b)); }, a.plan + 4 + a.pp);
}

// Launch of a kernel that may start while its predecessor in the stream still runs; it waits with pdl_wait() before
// it reads anything that the predecessor wrote.  pdl_trigger() in the predecessor lets it start.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Dynamic shared memory above 48 KB, allowed once per kernel and device.
template <typename... P> cudaError_t allow_smem(void (*kernel)(P...), size_t bytes) {
  static std::atomic<const void*> done[kMaxDevices];  // per kernel type and device: the last kernel allowed
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  const void* k = reinterpret_cast<const void*>(kernel);
  if (done[dev].load(std::memory_order_relaxed) == k) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e == cudaSuccess) done[dev].store(k, std::memory_order_relaxed);
  return e;
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

struct WeightsArgs {
  const void* K;
  const void* Q;
  const float* lse;      // [m][hq]
  const float* acc_in;   // NULL: zeros
  float* acc_out;        // [hkv][ld_acc_out]
  float* sums;           // partial column sums: [rsplit][hkv][n] (rsplit > 1), tensor cores: [CTA][2][256], then [hkv][n]
                         // for sums in place
  const float* logits;   // [hkv][rows][ld_logits] as the attention left them (NULL: computed again)
  int64_t ld_logits;
  int* status;           // NULL: no kernel of the call waits (fp32)
  int64_t ld, n, ld_acc_in, ld_acc_out;
  int rows;              // m * group
  int m, hq, hkv, group, causal, rsplit;
  int64_t rows_per_split;  // rows of one split (a multiple of the kernel's row block)
  float scale;
  long long wait_limit;  // bound of the waits on copies and products, SM cycles
};

// Host side: the plan of a call (kernel variant, CTAs, partial rows).
struct RowsPlan {
  int rb_log, kt_log, extra, nc, pp, po, rp, ro, rt;
  double places;  // most places the flat list can have
  uint64_t part_rows, part_own, part_tmp;
};
void rows_plan(int dtype, int d, int hkv, int group, int64_t B, int64_t m, int64_t n, int64_t ld_own, RowsPlan* p);
uint64_t rows_part_bound(int dtype, int d, int hkv, int group, int64_t B, int64_t m, int64_t n, int64_t ld_own);
void tc_plan(int64_t rows, int64_t mg, int64_t ld_own, RowsPlan* p);
cudaError_t launch_rows_tc(const RowsArgs& a, int d, cudaStream_t st);
cudaError_t launch_rows(const RowsArgs& a, int dtype, int d, cudaStream_t st);

struct WeightsPlan {
  int rsplit;
  int64_t rows_per_split;
  uint64_t sum_floats;  // partial sums in the scratch
  double places;        // places of the tensor-core kernel's list
};
void weights_plan(int dtype, int d, int hkv, int64_t rows, int64_t n, WeightsPlan* p);
uint64_t weights_sums_bound(int dtype, int hkv, int64_t n);
uint64_t weights_tc_floats();
cudaError_t launch_weights_tc(const WeightsArgs& a, int d, cudaStream_t st);
cudaError_t launch_weights(const WeightsArgs& a, int dtype, int d, cudaStream_t st);

// Calls of up to this many rows per KV head keep their logits (4 bytes per row and key) rather than read K again (2 d
// bytes per key) and run its products again.  Both sides, with outputs, 4 KV heads, us (kept / again):
//   bf16, 512K tokens   8 rows    16 rows   32 rows   64 rows      fp32     8 rows       16 rows      64 rows
//     d = 64            237/327   264/325   291/311   439/332              382/547      884/1123     1056/1485
//     d = 128           255/392   285/396   351/390   488/380              769/1607     1165/1836    2400/3538
// (64K tokens, bf16, d = 64: 50/65, 53/66, 58/67, 91/68).  Above 16 rows the gain of bf16 shrinks while the workspace
// grows with the rows, 128 bytes per key at 32; fp32 would gain on, for the same memory.
constexpr int kLogitRows = 16;

struct EvictArgs {
  const void* K;
  const void* V;
  const float* acc;
  void* K_out;
  void* V_out;
  float* acc_out;
  int32_t* idx;           // [hkv][keep]
  void* scratch;          // evict_scratch_bytes (long caches)
  int64_t ld, ld_acc, ld_out, ld_acc_out, n, keep, first, last;
  int hkv, row_bytes;     // bytes of one token's row of K or V
  int in_place;           // some output is its own input: rows move in order
};
uint64_t evict_scratch_bytes(int hkv, int64_t n);
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st);

}  // namespace zha
