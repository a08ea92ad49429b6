// Rows moved inside the paged grouped-query cache: the accepted path of a drafted tree brought
// together behind the cached tokens (compact), and requests that continue another one's tokens in
// pages of their own (fork). The cache is laid out as in kv_append.cu: [page, KV head, slot, d].
#include <cfloat>
#include <cstdint>

#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tts {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

// ---- compact -----------------------------------------------------------------------------
// A request's path keeps its new tokens path[0] < path[1] < .. of those behind `past`; row
// past + path[i] goes to past + i. Rows before the first with path[i] > i stay.
//
// A warp per (request, head, K or V) holds the rows in registers between all reads and the first
// write: up to 16 pieces of 16 bytes a lane (64 rows of 128 bytes; longer bf16 paths go in two
// batches, which is safe in order, since a later source lies behind every earlier destination).
// Lane i looks up rows i and i + 32: whatever the path's length, lengths and path are one round of
// loads, table entries the second, rows (e4m3: the pages' scales, then rows) the last, and there is no
// barrier but the warp's.
//
// e4m3: a page's scale holds for all of its slots. Where the rows moved into a page need a larger
// one, it becomes the smallest power of two that holds them and every code of the page moves with it.
//
// Measured (CUDA graph): 8 requests of e4m3 4.8 us, 256 of bf16 (15 MB read and written) 6.3 us for 2.2 us of
// bytes at the rate of a copy; those rounds, each of which waits for the one before, and the launch are
// what is left.
struct CompactParams {
  uint8_t* cache[2];  // K, V
  float* scale[2];
  const int32_t* page_tables;
  const int32_t* past;
  const int32_t* path;
  const int32_t* path_lens;
  int32_t* kv_lens;
  uint32_t* dev_status;
  int num_pages, hkv, page_shift, max_pages, batch, max_path;
};

// 16 codes times a factor, rounded to e4m3 again.
__device__ __forceinline__ uint4 rescale16(const uint4& v, float f) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3x2_to_float2((uint16_t)w[i]), b = e4m3x2_to_float2((uint16_t)(w[i] >> 16));
    w[i] = cvt_e4m3x2(a.x * f, a.y * f) | (cvt_e4m3x2(b.x * f, b.y * f) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Largest finite |value| of 16 codes.
__device__ __forceinline__ float amax16(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3x2_to_float2((uint16_t)w[i]), b = e4m3x2_to_float2((uint16_t)(w[i] >> 16));
    m = fmaxf(fmaxf(m, fmaxf(finite_abs(a.x), finite_abs(a.y))),
              fmaxf(finite_abs(b.x), finite_abs(b.y)));
  }
  return m;
}

template <int kCpr, bool kF8>  // pieces of 16 bytes per row
__global__ void __launch_bounds__(256) compact_kernel(const CompactParams p) {
  constexpr int kHold = 16;                      // pieces a lane holds
  constexpr int kBatchRows = kHold * 32 / kCpr;  // rows of a batch
  static_assert(!kF8 || kBatchRows >= 64, "e4m3 rows are held all at once");
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int r = (int)(w / (2 * p.hkv));
  if (r >= p.batch) return;
  const int hh = (int)(w % (2 * p.hkv));
  const bool is_v = hh >= p.hkv;
  const int h = is_v ? hh - p.hkv : hh;
  const bool first = hh == 0;  // reports, and writes the length
  float* const scales = is_v ? p.scale[1] : p.scale[0];
  const int past = p.past[r];
  int m = p.path_lens[r];
  int at[2];  // path of rows lane and lane + 32
#pragma unroll
  for (int k = 0; k < 2; ++k)
    at[k] = lane + 32 * k < p.max_path ? p.path[(int64_t)r * p.max_path + lane + 32 * k] : -1;
  uint32_t bad = 0;
  if (m < 0 || m > p.max_path) {
    bad = kDevBadArg;
    m = 0;
  }
  {
    const int up0 = __shfl_up_sync(kAll, at[0], 1), up1 = __shfl_up_sync(kAll, at[1], 1);
    const int top0 = __shfl_sync(kAll, at[0], 31);
    const bool wrong = (lane < m && at[0] <= (lane > 0 ? up0 : -1)) ||
                       (lane + 32 < m && at[1] <= (lane > 0 ? up1 : top0));
    if (__any_sync(kAll, wrong)) bad |= kDevBadArg;
  }
  const int last0 = __shfl_sync(kAll, at[0], (m - 1) & 31), last1 = __shfl_sync(kAll, at[1], (m - 1) & 31);
  // in 64 bits: a path's entries may be any int
  const int64_t last = m == 0 ? -1 : m > 32 ? last1 : last0, end = past + last + 1;
  if (past < 0 || end > ((int64_t)p.max_pages << p.page_shift)) bad |= kDevIndexRange;
  if (first && lane == 0) {
    p.kv_lens[r] = bad ? (past > 0 ? past : 0) : past + m;
    if (bad && p.dev_status != nullptr) atomicOr(p.dev_status, bad);
  }
  if (bad) return;
  const uint32_t same0 = __ballot_sync(kAll, lane < m && at[0] == lane);
  const uint32_t same1 = __ballot_sync(kAll, lane + 32 < m && at[1] == lane + 32);
  const int f = __popc(same0) + __popc(same1);  // strictly increasing: they come first
  if (f == m) return;
  const int slots = 1 << p.page_shift;
  int64_t from[2], to[2];                        // cache rows, -1: this row is not moved
  [[maybe_unused]] float s_from[2] = {1.f, 1.f}, s_to[2] = {1.f, 1.f};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    from[k] = to[k] = -1;
    if (i < f || i >= m) continue;
    const int src = past + at[k], dst = past + i;
    const int32_t* table = p.page_tables + (int64_t)r * p.max_pages;
    const int ps = table[src >> p.page_shift], pd = table[dst >> p.page_shift];
    if (ps < 0 || ps >= p.num_pages || pd < 0 || pd >= p.num_pages) {
      bad |= kDevIndexRange;
      continue;
    }
    const int64_t ss = (int64_t)ps * p.hkv + h, sd = (int64_t)pd * p.hkv + h;
    if constexpr (kF8) {
      s_from[k] = scales[ss];
      s_to[k] = scales[sd];
      if (!(s_from[k] > 0.f && s_from[k] < INFINITY)) {  // no scale a cached row can have
        bad |= kDevBadArg;
        continue;
      }
      if (!(s_to[k] > 0.f && s_to[k] < INFINITY)) {  // the page holds nothing: it is begun here
        bad |= kDevBadArg;
        s_to[k] = 0.f;
      }
    }
    from[k] = (ss << p.page_shift) + (src & (slots - 1));
    to[k] = (sd << p.page_shift) + (dst & (slots - 1));
  }
  if (bad && p.dev_status != nullptr) atomicOr(p.dev_status, bad);
  uint4* const rows = reinterpret_cast<uint4*>(is_v ? p.cache[1] : p.cache[0]);
  auto row64 = [&](const int64_t (&x)[2], int i) -> int64_t {  // x of row i (lane-varying)
    const int64_t a = __shfl_sync(kAll, x[0], i & 31), b = __shfl_sync(kAll, x[1], i & 31);
    return i < 32 ? a : b;
  };
  auto rowf = [&](const float (&x)[2], int i) -> float {
    const float a = __shfl_sync(kAll, x[0], i & 31), b = __shfl_sync(kAll, x[1], i & 31);
    return i < 32 ? a : b;
  };
  // e4m3: page by page. A later page's sources lie behind this page, so that its codes may move to a new
  // scale once the rows that come into it are read.
  for (int b0 = f, b1; b0 < m; b0 = b1) {
    b1 = min(m, kF8 ? (((past + b0) >> p.page_shift) + 1 << p.page_shift) - past : b0 + kBatchRows);
    const int pieces = (b1 - b0) * kCpr;
    uint4 held[kHold];
    float top = 0.f;  // largest value that comes into the page
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      held[k] = make_uint4(0, 0, 0, 0);
      if (k * 32 >= pieces) continue;  // the same for the warp
      const int x = k * 32 + lane;
      const int64_t src = row64(from, b0 + x / kCpr);
      if (x < pieces && src >= 0) held[k] = rows[src * kCpr + x % kCpr];
    }
    __syncwarp();  // all rows are read before any is written
    [[maybe_unused]] float scale = 1.f;
    if constexpr (kF8) {
#pragma unroll
      for (int k = 0; k < kHold; ++k)
        if (k * 32 < pieces) {
          const float s = rowf(s_from, b0 + (k * 32 + lane) / kCpr);
          top = fmaxf(top, amax16(held[k]) * s);  // rows that are not moved are held as zeros
        }
      top = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(top)));
      // a row that is moved tells the page
      const uint32_t in0 = __ballot_sync(kAll, lane >= b0 && lane < b1 && to[0] >= 0);
      const uint32_t in1 = __ballot_sync(kAll, lane + 32 >= b0 && lane + 32 < b1 && to[1] >= 0);
      if ((in0 | in1) == 0) continue;
      const int i = in0 ? __ffs(in0) - 1 : 31 + __ffs(in1);
      const int64_t slab = row64(to, i) >> p.page_shift;
      const float old = rowf(s_to, i);
      scale = old;
      if (!(old > 0.f && top <= 448.f * old)) {
        scale = block_scale(top);
        uint4* at = rows + (slab << p.page_shift) * kCpr;
        if (old > 0.f)
          for (int x = lane; x < slots * kCpr; x += 32) at[x] = rescale16(at[x], old / scale);
        if (lane == 0) scales[slab] = scale;
        __syncwarp();  // rows are written over a page that has its new codes
      }
    }
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      if (k * 32 >= pieces) continue;
      const int x = k * 32 + lane;
      const int64_t dst = row64(to, b0 + x / kCpr);
      if constexpr (kF8) {
        const float s = rowf(s_from, b0 + x / kCpr);
        // finite also where scales lie further apart than fp32 reaches: such a row is zeros
        if (s != scale) held[k] = rescale16(held[k], fminf(s / scale, FLT_MAX));
      }
      if (x < pieces && dst >= 0) rows[dst * kCpr + x % kCpr] = held[k];
    }
    __syncwarp();
  }
}

// ---- fork --------------------------------------------------------------------------------
// New request i continues request parents[i]: its table row is the parent's up to the last full
// page, its last, partly filled page is new_pages[i] with the parent's rows (and scales) in it.
//
// A block per (new request, head) copies the used rows of a page's K and V, one more per request
// writes the table row and the length.
//
// Bound: HBM for many beams (CUDA graph, 512 of them in bf16, 33 MB read and 33 written: 11.8 us for
// 9.8 at the rate of a copy), a launch and one chain of loads for few (4 samples in e4m3: 2.3 us).
struct ForkParams {
  uint4* cache[2];
  float* scale[2];  // null: bf16
  const int32_t* page_tables;
  const int32_t* kv_lens;
  const int32_t* parents;
  const int32_t* new_pages;
  int32_t* tables_out;
  int32_t* lens_out;
  uint32_t* dev_status;
  int num_pages, hkv, page_shift, max_pages, batch, cpr;
};

constexpr int kForkThreads = 128;
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const ForkParams p) {
  wait_for_prior_grids();
  const int tid = threadIdx.x;
  const int i = (int)(blockIdx.x / (p.hkv + 1)), part = (int)(blockIdx.x % (p.hkv + 1));
  const int parent = p.parents[i];
  const int fresh = p.new_pages[i];
  uint32_t bad = 0;
  int len = 0;
  if (parent < 0 || parent >= p.batch) {
    bad = kDevIndexRange;
  } else {
    len = p.kv_lens[parent];
    if (len < 0 || (int64_t)len > ((int64_t)p.max_pages << p.page_shift)) {
      bad = kDevIndexRange;
      len = 0;
    }
  }
  const int full = len >> p.page_shift, used = len & ((1 << p.page_shift) - 1);
  const int32_t* old = p.page_tables + (int64_t)(bad ? 0 : parent) * p.max_pages;
  if (fresh >= p.num_pages) bad |= kDevIndexRange;
  const bool own = fresh >= 0 && fresh < p.num_pages;  // else the parent's row is shared whole
  if (part == p.hkv) {
    int32_t* t = p.tables_out + (int64_t)i * p.max_pages;
    const bool none = parent < 0 || parent >= p.batch || (bad && len == 0);
    for (int x = tid; x < p.max_pages; x += kForkThreads) {
      int v = -1;
      if (!none) {
        if (x < full || !own)
          v = fresh >= p.num_pages && x >= full ? -1 : old[x];
        else if (x == full)
          v = fresh;
      }
      t[x] = v;
    }
    if (tid == 0) p.lens_out[i] = len;
    if (tid == 0 && used > 0 && own && !bad) {
      const int src = old[full];
      if (src < 0 || src >= p.num_pages) bad |= kDevIndexRange;
    }
    if (tid == 0 && bad && p.dev_status != nullptr) atomicOr(p.dev_status, bad);
    return;
  }
  if (bad || !own || used == 0) return;
  const int src = old[full];
  if (src < 0 || src >= p.num_pages || src == fresh) return;
  const int64_t from = (int64_t)src * p.hkv + part, to = (int64_t)fresh * p.hkv + part;
  const int64_t at_from = (from << p.page_shift) * p.cpr, at_to = (to << p.page_shift) * p.cpr;
  if (tid == 0 && p.scale[0] != nullptr) {
    p.scale[0][to] = p.scale[0][from];
    p.scale[1][to] = p.scale[1][from];
  }
  const int n = used * p.cpr;
  constexpr int kDeep = 4;
  for (int x0 = 0; x0 < n; x0 += kForkThreads * kDeep) {
    uint4 v[2][kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int x = x0 + k * kForkThreads + tid;
      if (x < n) {
        v[0][k] = p.cache[0][at_from + x];
        v[1][k] = p.cache[1][at_from + x];
      }
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int x = x0 + k * kForkThreads + tid;
      if (x < n) {
        p.cache[0][at_to + x] = v[0][k];
        p.cache[1][at_to + x] = v[1][k];
      }
    }
  }
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

}  // namespace

cudaError_t launch_kv_compact(const KvCompactArgs& a, cudaStream_t stream) {
  CompactParams p;
  p.cache[0] = static_cast<uint8_t*>(a.cache.k);
  p.cache[1] = static_cast<uint8_t*>(a.cache.v);
  p.scale[0] = a.cache.k_scale;
  p.scale[1] = a.cache.v_scale;
  p.page_tables = a.page_tables;
  p.past = a.past_lens;
  p.path = a.path;
  p.path_lens = a.path_lens;
  p.kv_lens = a.kv_lens;
  p.dev_status = a.dev_status;
  p.num_pages = a.cache.num_pages;
  p.hkv = a.cache.hkv;
  p.page_shift = log2_of(a.cache.page_size);
  p.max_pages = a.max_pages;
  p.batch = a.batch;
  p.max_path = a.max_path;
  const int64_t warps = (int64_t)a.batch * 2 * a.cache.hkv;
  const int64_t blocks = (warps + 7) / 8;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks);
  const int row = a.cache.d * (a.cache.f8 ? 1 : 2);
  if (a.cache.f8)
    return row == 128 ? launch_ahead(compact_kernel<8, true>, grid, 256, 0, stream, p)
                      : launch_ahead(compact_kernel<4, true>, grid, 256, 0, stream, p);
  return row == 256 ? launch_ahead(compact_kernel<16, false>, grid, 256, 0, stream, p)
                    : launch_ahead(compact_kernel<8, false>, grid, 256, 0, stream, p);
}

cudaError_t launch_kv_fork(const KvForkArgs& a, cudaStream_t stream) {
  ForkParams p;
  p.cache[0] = static_cast<uint4*>(a.cache.k);
  p.cache[1] = static_cast<uint4*>(a.cache.v);
  p.scale[0] = a.cache.f8 ? a.cache.k_scale : nullptr;
  p.scale[1] = a.cache.f8 ? a.cache.v_scale : nullptr;
  p.page_tables = a.page_tables;
  p.kv_lens = a.kv_lens;
  p.parents = a.parents;
  p.new_pages = a.new_pages;
  p.tables_out = a.tables_out;
  p.lens_out = a.lens_out;
  p.dev_status = a.dev_status;
  p.num_pages = a.cache.num_pages;
  p.hkv = a.cache.hkv;
  p.page_shift = log2_of(a.cache.page_size);
  p.max_pages = a.max_pages;
  p.batch = a.batch;
  p.cpr = a.cache.d * (a.cache.f8 ? 1 : 2) / 16;
  const int64_t blocks = (int64_t)a.children * (a.cache.hkv + 1);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_ahead(fork_kernel, dim3((unsigned)blocks), kForkThreads, 0, stream, p);
}

}  // namespace tts
