// Attention of the newest tokens of each request over a paged grouped-query KV cache held in
// e4m3 (a scale per page and KV head) or bf16, with an optional sliding window and first
// tokens that stay visible.
//
// For KV head g the q rows of its group (token-major: row = token * G + head in the group)
// are tiles of 8 to 64 rows; a unit is (request, g, row tile) and a tile is kTK consecutive keys.
// With x_j = scale log2(e) sK[page(j)] q.k_j (q.k over codes), y_j = x_j + log2 sV[page(j)]:
//   out = sum_j 2^(y_j - m) v_j / sum_j 2^(y_j - m) / sV[page(j)],  lse = ln 2 (m + log2 of the
// denominator): the value scale rides in the exponent, so weights of pages with different
// scales share one fp16 product with the codes, and the running maximum m is taken over y.
//
// Bound: HBM (a cached byte is used by a unit's few rows only). All tiles of all units form one
// list, cut into equal runs, one per CTA (two CTAs per SM), so ragged batches, one request and
// many requests all fill the GPU; a unit cut by a run's border leaves unnormalised partial
// sums, joined in a fixed order by a second launch. In a CTA one warp brings tiles by TMA
// (pages through the table, 128-byte swizzle) into a ring of kStages slots, and each of four
// warps takes every fourth tile for itself, with its own running maximum, sum and
// accumulators, joined through shared memory at the end of the unit: no barrier inside a unit.
//
// S^T = K Q^T and O^T = V^T P^T run on m16n8k16 tensor-core products with keys (then d) as the 16
// rows and q rows as the 8 columns: a group of 4 to 8 heads fills the columns, and a warp takes
// its operands from shared memory into registers, where e4m3 is widened; at HBM's rate an SM can
// issue about 2800 instructions per 16 KB tile, of which one n tile takes a third (issue slots 29
// % used, tensor pipe 18 %), so that up to 8 rows the bytes are the bound. More rows repeat the
// loads and the widening of a tile in each row group: there tcgen05 products with 128 keys (then
// d) as rows and the q rows as columns would take a tile once. They are not built. e4m3 codes
// become fp16 (exactly) in registers; q is fp16 after a power-of-two scaling of its row (exact for
// every element within 2^-22 of the row's largest), and P is fp16 with its reference kept so that
// 2^-25 of the maximum still has all 11 bits. bf16 caches use bf16 products throughout. Sums and
// softmax statistics are fp32.
//
// Measured (32 / 8 heads of 128; from one GPU to another): 64 requests x 32768 tokens in e4m3 616
// to 636 us (6.8 to 7.0 TB/s, 1.00 to 1.03 of the measured copy rate), one request of 2590 tokens
// 8.5 to 9.7 us (the chain of launch, lengths, page table, tile, products and the parts' launch;
// its bytes are 0.8 us), 33 ragged requests with a window of 4096 53 us (39.4 us of bytes; about
// 2.5 us before the first tile, 3 for the parts, and the last CTAs), 1 to 4 tokens of 16 requests
// over a bf16 cache 64 to 66 us (52.7). Many rows are bound by what each warp issues: 8, 16, 32
// and 64 rows per KV head take 1.2, 1.6, 2.2 and 3.7 times the bytes' time in e4m3 and 1.1, 1.1,
// 1.3 and 2.0 in bf16 (16 requests x 20000 tokens, 4 KV heads; CUDA graph).
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tts {
namespace {

constexpr int kNW = 4;                        // consumer warps
constexpr int kThreads = (kNW + 1) * 32;      // and one producer warp
constexpr int kCtasPerSm = 2;
// What the end of a unit costs (joining the warps, the next unit's q), in tiles: the list that
// is cut into runs has this many empty places behind a unit's tiles, so that a run over many
// short units is not the last to finish (33 ragged requests, window 4096, pages of 64: 57.9 us
// without, 51.8 with).
constexpr int kEndTiles = 3;
// Smallest value scale: a key adds a weight of at most 2^15 over its scale to the denominator, which
// for 2^30 keys then stays under 2^125. The append writes none below 2^-60.
constexpr float kMinValueScale = 0x1p-80f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// NT: 8-row n tiles of a warp. kGroups: a request with more than 8 NT rows per KV head has them
// worked on by 2 or 4 row groups of warps on the same tiles of keys (which are then read once for
// up to 32 NT rows), one with fewer by all warps on different tiles.
template <bool F8, int D, int NT>
struct Cfg {
  static constexpr int kRowBytes = D * (F8 ? 1 : 2);
  static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;  // one swizzled TMA box row
  static constexpr int kPanels = kRowBytes / kPanelBytes;
  // Keys per tile: 16 KB of K and V together, so that the producer's work per tile is a small
  // part of the time its bytes take, but no more than 64 keys' scores in registers with two n
  // tiles (64-wide e4m3 rows, 20,000 keys: 8 KB tiles 46.5 us, 16 KB tiles 36.7 us).
  static constexpr int kTK = kRowBytes == 256 ? 32 : kRowBytes == 64 && NT == 1 ? 128 : 64;
  static constexpr int kMT = kTK / 16;
  // m tiles whose scores are in registers together: with two n tiles two, in passes over the
  // tile. Shared memory leaves little of L1, so every register spilled is read from L2 (16 q
  // rows, 16 x 20,000 keys of e4m3: 85 us with four m tiles, 77 with two and the room below).
  static constexpr int kPass = NT == 2 ? 2 : kMT;
  static constexpr int kKBytes = kTK * kRowBytes;  // K (or V) of one tile
  static constexpr int kStageBytes = 2 * kKBytes;
  static constexpr int kGR = 8 * NT;       // q rows per row group
  static constexpr int kKS = D / 16;       // k steps of the first product, m tiles of the second
  static constexpr int kPieces = kTK / 16;  // pages of a tile at most
  static constexpr int kQStride = D * 2 + 16;  // bytes per q row in shared memory (two n tiles)
  // Behind the ring: the warps' accumulators on their way to the one that sums them, and the q
  // rows of RG row groups. They share the room: RG groups leave 1 / RG of the warps to join.
  template <int RG>
  static constexpr int join_bytes() {
    return kNW * (kNW / RG - 1) * NT * (kKS * RG / kNW) * 4 * 32 * 4;
  }
  template <int RG>
  static constexpr int room() {
    return join_bytes<RG>() + (NT > 1 ? RG * kGR * kQStride : 0);
  }
  static constexpr int kJoinBytes =
      room<1>() > room<2>() ? (room<1>() > room<4>() ? room<1>() : room<4>())
                            : (room<2>() > room<4>() ? room<2>() : room<4>());
  // Two CTAs per SM: 113 KB each, less 1 KB to align the ring and 1 KB of barriers.
  static constexpr int kStagesFit = (113 * 1024 - 2048 - kJoinBytes) / kStageBytes;
  // Two n tiles leave 16 KB to L1: their spilled registers are read from it.
  static constexpr int kStages =
      (kStagesFit < 12 ? kStagesFit : 12) - (NT == 2 ? 16384 / kStageBytes : 0);
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kJoinBytes;
};

struct Params {
  const uint16_t* q;
  const int32_t* cu_q;  // null: one token per request
  const int32_t* page_tables;
  const int32_t* kv_lens;
  const float* k_scale;
  const float* v_scale;
  void* out;
  float* lse;
  float* parts;  // [2 * CTAs][unit_rows * (D + 2)]
  // [CTAs], of the unit that was begun in an earlier CTA and ended in this one: {first CTA
  // (-1: no such unit), rows, first row within the request, g}
  int4* jobs;
  int* job_q0;  // and the request's first q row
  uint32_t* dev_status;
  int total_q, max_keys;
  int batch, max_q, hq, hkv, group, num_pages, max_pages, page_size, page_shift, window, sinks;
  float scale_log2;
  int out_bf16, ctas, unit_rows, row_shift;  // a unit's q rows (a power of two)
};

// A request as the kernel sees it: its tokens, its visible keys as two runs of tiles (first
// tokens, window) and the number of units per head.
struct Req {
  int n, L, lo, sinks;  // new tokens, keys, first key of the window (0: none), kept first keys
  int st, lt, nt, rt;   // tiles of the first keys, first tile of the window, tiles, row tiles
  int q0;               // first q row
};
__device__ __forceinline__ void read_req(const Params& p, int b, int& n, int& L, int& q0,
                                         uint32_t* bad) {
  int q1 = b + 1;
  q0 = b;
  if (p.cu_q != nullptr) {
    q0 = p.cu_q[b];
    q1 = p.cu_q[b + 1];
  }
  L = p.kv_lens[b];
  n = 0;
  if (q0 < 0 || q1 < q0 || q1 > p.total_q || q1 - q0 > p.max_q)
    *bad |= kDevBadArg;
  else
    n = q1 - q0;
  if (L < 0 || L > p.max_keys) {
    *bad |= kDevIndexRange;
    L = 0;  // its rows see no key
  }
}
template <int TK>
__device__ __forceinline__ Req make_req(const Params& p, int n, int L, int q0) {
  Req r;
  r.n = n;
  r.L = L;
  r.q0 = q0;
  // keys and window are at most 2^30, so nothing here leaves 32 bits
  r.lo = p.window > 0 ? max(L - n + 1 - p.window, 0) : 0;
  r.sinks = min(p.sinks, r.lo);
  r.lt = (int)((unsigned)r.lo / TK);
  r.st = min((int)((unsigned)(r.sinks + TK - 1) / TK), r.lt);
  r.nt = max(r.st + (int)((unsigned)(L + TK - 1) / TK) - r.lt, 1);  // 1: an empty tile, zeros
  r.rt = (n * p.group + p.unit_rows - 1) >> p.row_shift;
  return r;
}
template <int TK>
__device__ __forceinline__ Req load_req(const Params& p, int b, uint32_t* bad) {
  int n, L, q0;
  read_req(p, b, n, L, q0, bad);
  return make_req<TK>(p, n, L, q0);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool F8>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  if constexpr (F8)
    mma_f16(d, a, b0, b1);
  else
    mma_bf16(d, a, b0, b1);
}
// 8x8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The two e4m3 codes in the low / high half of w as two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}

// Shared-memory address of 16-byte chunk c of row `row` of a K or V tile, as TMA's swizzle
// places it (128-byte rows: chunk ^ row mod 8; 64-byte rows: chunk ^ row / 2 mod 4).
template <int TK, int PB>
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int row, int c) {
  if constexpr (PB == 128)
    return base + (c >> 3) * (TK * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  else
    return base + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

template <int kP>
struct Meta {  // of a ring slot, written by the producer
  uint32_t ok;   // bit i: piece i of the tile (a page, or the tile if pages are larger) is there
  float ks[kP];  // scale of its keys
  float vl[kP];  // log2 of the scale of its values
  float vi[kP];  // 1 / that scale
};

template <bool F8, int D, int NT, bool kGroups>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    attn_decode_kernel(const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const Params p) {
  using C = Cfg<F8, D, NT>;
  constexpr int TK = C::kTK, MT = C::kPass, S = C::kStages, KS = C::kKS, GR = C::kGR;
  // Releases of a ring slot: the one warp that worked on it, or with row groups every warp.
  constexpr int kReleases = kGroups ? kNW : 1;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[S], bar_empty[S];
  __shared__ Meta<F8 ? C::kPieces : 1> s_meta[S];
  __shared__ __align__(8) float s_m[kNW][GR], s_l[kNW][GR];  // references and sums of every row
  __shared__ int s_scan[kThreads / 32], s_b, s_off, s_abort, s_issued;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* join = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)) + S * C::kStageBytes);
  volatile int* abort_flag = &s_abort;
  volatile int* issued_tiles = &s_issued;

  if (tid == kNW * 32) {  // on their way while the lengths are read
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  wait_for_prior_grids();
  // ---- this CTA's run [t0, t1) of the list of tiles, and the request it begins in
  uint32_t bad = 0;
  if (tid == 0) {
    s_abort = s_issued = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&bar_full[i]), 1);
      mbar_init(smem_u32(&bar_empty[i]), kReleases);
    }
    fence_mbar_init();
    p.jobs[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  auto scan32 = [&](int x) -> int {  // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  auto tiles_of = [&](const Req& r) -> int { return p.hkv * r.rt * (r.nt + kEndTiles); };
  // One run per kNW places of the list, rounded up (the warps take one each, side by side): shorter
  // runs would only leave more parts to join. The first `more` runs have one place more than the
  // others; rounding may leave a run of a short list a place or two under kNW.
  int total = 0, runs = 0, len = 0, more = 0, t0 = 0, t1 = 0;
  auto split = [&]() -> bool {
    runs = min((int)((unsigned)(total + kNW - 1) / kNW), p.ctas);
    if ((int)blockIdx.x >= runs) return false;
    len = (int)((unsigned)total / (unsigned)runs);
    more = total - len * runs;
    t0 = blockIdx.x * len + min((int)blockIdx.x, more);
    t1 = t0 + len + ((int)blockIdx.x < more ? 1 : 0);
    return true;
  };
  int b = 0, off = 0;
  Req r;
  if (p.batch <= 32) {  // every warp for itself
    int n = 0, L = 0, q0 = 0, v = 0;
    if (lane < p.batch) {
      read_req(p, lane, n, L, q0, &bad);
      r = make_req<TK>(p, n, L, q0);
      v = tiles_of(r);
    }
    if (blockIdx.x == 0 && warp == 0 && bad && p.dev_status != nullptr)
      atomicOr(p.dev_status, bad);
    const int incl = scan32(v);
    total = __shfl_sync(0xFFFFFFFFu, incl, 31);
    if (!split()) return;
    b = __ffs(__ballot_sync(0xFFFFFFFFu, incl > t0)) - 1;
    off = t0 - __shfl_sync(0xFFFFFFFFu, incl - v, b);
    r = make_req<TK>(p, __shfl_sync(0xFFFFFFFFu, n, b), __shfl_sync(0xFFFFFFFFu, L, b),
                        __shfl_sync(0xFFFFFFFFu, q0, b));
  } else {
    auto block_scan = [&](int v, int* sum) -> int {  // inclusive
      const int x = scan32(v);
      __syncthreads();
      if (lane == 31) s_scan[warp] = x;
      __syncthreads();
      int before = 0;
      *sum = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        *sum += s_scan[w];
      }
      return x + before;
    };
    for (int base = 0; base < p.batch; base += kThreads) {
      const int i = base + tid;
      int sum;
      block_scan(i < p.batch ? tiles_of(load_req<TK>(p, i, &bad)) : 0, &sum);
      total += sum;
    }
    if (blockIdx.x == 0 && bad && p.dev_status != nullptr) atomicOr(p.dev_status, bad);
    if (!split()) return;
    for (int base = 0, carry = 0; base < p.batch && carry <= t0; base += kThreads) {
      const int i = base + tid;
      const int v = i < p.batch ? tiles_of(load_req<TK>(p, i, &bad)) : 0;
      int sum;
      const int incl = carry + block_scan(v, &sum);
      if (incl > t0 && incl - v <= t0) {
        s_b = i;
        s_off = t0 - (incl - v);
      }
      carry += sum;
    }
    __syncthreads();
    b = s_b;
    off = s_off;
    r = load_req<TK>(p, b, &bad);
  }
  __syncthreads();

  int left = t1 - t0;
  int it = 0;  // tiles of this run so far
  int seg_g = -1, seg_rt = 0;
  // The next unit's part in this run: head, row tile, tiles [x0, x1) of nt.
  auto next_seg = [&](int& g, int& rt, int& x0, int& x1) -> bool {
    if (seg_g < 0) {  // the run's first unit, perhaps from its middle
      const int u = (int)((unsigned)off / (unsigned)(r.nt + kEndTiles));
      x0 = off - u * (r.nt + kEndTiles);
      seg_g = (int)((unsigned)u / (unsigned)r.rt);
      seg_rt = u - seg_g * r.rt;
    } else {
      x0 = 0;
      if (++seg_rt == r.rt) {
        seg_rt = 0;
        if (++seg_g == p.hkv) {
          seg_g = 0;
          do r = load_req<TK>(p, ++b, &bad);  // requests without new tokens have no units
          while (r.rt == 0);
        }
      }
    }
    g = seg_g;
    rt = seg_rt;
    x1 = min(r.nt, x0 + left);
    left -= min(r.nt + kEndTiles - x0, left);
    return x0 < x1;  // else the run begins behind the unit's last tile
  };
  const int piece = p.page_size < TK ? p.page_size : TK;  // keys per TMA box
  const int n_pieces = TK / piece;

  if (warp == kNW) {
    // ------------------------------------------------------------------ producer
    // A tile must leave in well under the ~700 cycles that HBM takes for it, so lane i keeps
    // page cache_at + i of the request (and what the consumers need of its scales for head
    // cache_g) in registers, loaded 32 pages at a time.
    constexpr uint32_t kBox = C::kPanelBytes;
    int cache_b = -1, cache_at = 0, cache_g = -1, page = -1;
    bool fine = true;                    // the page's scales are in range
    float ks = 1.f, vl = 0.f, vi = 1.f;  // key scale, log2 and inverse of the value scale
    bool ok = true;
    while (ok && left > 0) {
      int g, rt, x0, x1;
      if (!next_seg(g, rt, x0, x1)) continue;
      for (int x = x0; ok && x < x1; ++x, ++it) {
        const int key0 = (x < r.st ? x : r.lt + x - r.st) * TK;
        const int st = it % S;
        const int pg0 = key0 >> p.page_shift;
        if (cache_b != b || pg0 < cache_at || pg0 + n_pieces > cache_at + 32) {
          cache_b = b;
          cache_at = pg0;
          cache_g = -1;
          const int lp = pg0 + lane;
          page = lp < p.max_pages ? p.page_tables[(int64_t)b * p.max_pages + lp] : -1;
          if (page < 0 || page >= p.num_pages) page = -1;
        }
        float sk = 1.f, sv = 1.f;
        const bool new_scales = F8 && cache_g != g;
        if (new_scales && page >= 0) {  // asked for here, looked at behind the copies
          sk = p.k_scale[(int64_t)page * p.hkv + g];
          sv = p.v_scale[(int64_t)page * p.hkv + g];
        }
        const int at = pg0 - cache_at + (lane < n_pieces ? lane : 0);
        const int pg = __shfl_sync(0xFFFFFFFFu, page, at);
        const int a = key0 + lane * piece;  // this lane's piece: keys [a, a + piece)
        const bool seen = lane < n_pieces && a < r.L && (a + piece > r.lo || a < r.sinks);
        const bool there = seen && pg >= 0;
        const uint32_t sent = __ballot_sync(0xFFFFFFFFu, there);
        uint32_t flag = seen && !there ? kDevIndexRange : 0u;
        uint32_t use = sent;
        float pk = 1.f, pl = 0.f, pi = 1.f;
        auto scales = [&]() {
          const uint32_t all = __ballot_sync(0xFFFFFFFFu, fine);
          const bool good = there && ((all >> at) & 1u);
          if (there && !good) flag |= kDevBadArg;  // no scale of a written page: keys skipped
          use = __ballot_sync(0xFFFFFFFFu, good);
          // Pieces that are not used stay neutral: their page's scales may be anything (an inverse
          // of infinity times a weight of zero is NaN).
          const float k_of = __shfl_sync(0xFFFFFFFFu, ks, at), l_of = __shfl_sync(0xFFFFFFFFu, vl, at),
                      i_of = __shfl_sync(0xFFFFFFFFu, vi, at);
          pk = good ? k_of : 1.f;
          pl = good ? l_of : 0.f;
          pi = good ? i_of : 0.f;
        };
        if (F8 && !new_scales) scales();
        // All of the above may be done before the slot is free; little is left behind the wait.
        if (it >= S)
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&bar_empty[st]), ((it / S) - 1) & 1,
                                                 abort_flag, p.dev_status));
        if (!ok) break;
        const uint32_t bar = smem_u32(&bar_full[st]);
        if (there) {
          const uint32_t dst = ring + st * C::kStageBytes + lane * piece * kBox;
          const int row = key0 & (p.page_size - 1);  // 0 unless the tile is inside a page
          const int slab = pg * p.hkv + g;
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn) {
            tma_load_3d(dst + pn * TK * kBox, &map_k, bar, pn * 64, row, slab);
            tma_load_3d(dst + C::kKBytes + pn * TK * kBox, &map_v, bar, pn * 64, row, slab);
          }
        }
        if constexpr (F8) {
          if (new_scales) {
            cache_g = g;
            fine = sk > 0.f && sk < INFINITY && sv >= kMinValueScale && sv < INFINITY;
            ks = sk;
            vl = fine ? log2f(sv) : 0.f;
            vi = fine ? 1.f / sv : 0.f;
            scales();
          }
          if (lane < n_pieces) {
            s_meta[st].ks[lane] = pk;
            s_meta[st].vl[lane] = pl;
            s_meta[st].vi[lane] = pi;
          }
        }
        if (flag && p.dev_status != nullptr) atomicOr(p.dev_status, flag);
        if (lane == 0) s_meta[st].ok = use;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, __popc(sent) * piece * C::kRowBytes * 2);
          *issued_tiles = it + 1;
        }
      }
    }
    // Copies in flight must land before the CTA can exit, also when a consumer's wait ran out.
    for (int i = it > S ? it - S : 0; i < it; ++i)
      mbar_wait(smem_u32(&bar_full[i % S]), (i / S) & 1, nullptr, nullptr);
  } else {
    // ------------------------------------------------------------------ consumers
    constexpr float kThr = F8 ? 4.f : 8.f;    // the reference moves when exceeded by 2^kThr
    constexpr float kBias = F8 ? 11.f : 0.f;  // P is held times 2^kBias: at most 2^15 in fp16
    const int g8 = lane >> 2, t4 = lane & 3;
    const int piece_shift = 31 - __clz(piece >> 4);  // 16-key m tile -> piece
    // Bounded wait until the producer has issued tile i (usually long ago).
    auto issued = [&](int i) -> bool {
      bool ok = *issued_tiles > i;
      if (!ok) {
        const uint64_t since = globaltimer();
        while (!(ok = *issued_tiles > i) && !*abort_flag) {
          if (globaltimer() - since > kWaitLimitNs) {
            if (p.dev_status != nullptr) atomicOr(p.dev_status, kDevTimeout);
            *abort_flag = 1;
          }
        }
      }
      return __all_sync(0xFFFFFFFFu, ok);
    };
    // One unit's part in this run, its rows in RG groups.
    auto segment = [&](auto groups, int g, int rt, int x0, int x1, int before) {
      constexpr int RG = decltype(groups)::value;
      constexpr int GW = kNW / RG;  // warps per row group: each takes every GW-th tile
      constexpr int MQ = KS / GW;   // m tiles each warp finishes when the unit ends
      const int rg = warp / GW, wi = warp % GW;  // row group, place in it
      const bool whole_l = x0 == 0, whole_r = x1 == r.nt;
      // this row group's first row, and its rows: up to GR
      const int row0 = rt * p.unit_rows + rg * GR;
      const int rows = min(r.n * p.group - row0, GR);

      // q fragments of column g8 of every n tile: step i takes elements e0(i) .. e0(i) + 3. One n
      // tile's stay in registers; two n tiles' go to shared memory, once per row group, each row
      // as the products take it: step i's pairs of lanes 0 .. 3, then their second pairs.
      [[maybe_unused]] uint32_t qf[NT == 1 ? KS : 1][2];
      const uint32_t q_rows =
          smem_u32(join) + C::template join_bytes<RG>() + rg * (GR * C::kQStride);
      float f0[NT], f1[NT];      // factor of the scores of columns 2 t4 and 2 t4 + 1
      int pos0[NT], pos1[NT];    // positions of the two rows
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int rr = row0 + j * 8 + g8;
        const bool in = j * 8 + g8 < rows;
        const int tok = in && p.max_q > 1 ? rr / p.group : 0;
        const int h = in ? g * p.group + (rr - tok * p.group) : 0;
        const uint16_t* src = p.q + ((int64_t)(r.q0 + tok) * p.hq + h) * D;
        uint32_t w[KS][2];
#pragma unroll
        for (int i = 0; i < KS; i += 2) {
          const int e0 = F8 ? (D / 4) * t4 + 4 * i : 64 * (i / 4) + 16 * t4 + 4 * (i % 4);
          const uint4 v = in ? *reinterpret_cast<const uint4*>(src + e0) : make_uint4(0, 0, 0, 0);
          w[i][0] = v.x;
          w[i][1] = v.y;
          w[i + 1][0] = v.z;
          w[i + 1][1] = v.w;
        }
        float fac = p.scale_log2;
        if constexpr (F8) {
          uint32_t top = 0;  // largest |q| of the row, as bf16 bits
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t m = w[i][k] & 0x7FFF7FFFu;
              top = max(top, max(m & 0xFFFFu, m >> 16));
            }
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const int e = max((int)(top >> 7), 27);  // biased exponent; q' = q 2^(8 - e) < 2^9
          const float up = __uint_as_float((uint32_t)(262 - e < 1 ? 1 : 262 - e) << 23);
          fac *= __uint_as_float((uint32_t)(e < 9 ? 1 : e - 8) << 23);
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              w[i][k] = pack_f16x2(__uint_as_float(w[i][k] << 16) * up,
                                   __uint_as_float(w[i][k] & 0xFFFF0000u) * up);
        }
        if constexpr (NT == 1) {
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            qf[i][0] = w[i][0];
            qf[i][1] = w[i][1];
          }
        } else if (wi == 0) {
          const uint32_t to = q_rows + (j * 8 + g8) * C::kQStride + t4 * 4;
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + i * 32), "r"(w[i][0]) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + i * 32 + 16), "r"(w[i][1]) : "memory");
          }
        }
        const int pos = r.L - r.n + tok;
        f0[j] = __shfl_sync(0xFFFFFFFFu, fac, (2 * t4) * 4);
        f1[j] = __shfl_sync(0xFFFFFFFFu, fac, (2 * t4 + 1) * 4);
        pos0[j] = __shfl_sync(0xFFFFFFFFu, pos, (2 * t4) * 4);
        pos1[j] = __shfl_sync(0xFFFFFFFFu, pos, (2 * t4 + 1) * 4);
      }
      auto group_sync = [&]() {
        if constexpr (GW > 1)
          named_barrier_sync(RG + rg, GW * 32);
        else
          __syncwarp();
      };
      if constexpr (NT > 1) group_sync();  // q rows written
      // steps i and i + 1 of n tile j: b0, b1 of each
      auto q_frag = [&](int j, int i, uint32_t (&b)[4]) {
        if constexpr (NT == 1) {
          b[0] = qf[i][0];
          b[1] = qf[i][1];
          b[2] = qf[i + 1][0];
          b[3] = qf[i + 1][1];
        } else {
          ldsm_x4(b, q_rows + (j * 8 + (lane & 7)) * C::kQStride + i * 32 + (lane >> 3) * 16);
        }
      };
      // every row sees keys [max_lo, min_end) (and the first sinks)
      const int min_end = r.L - r.n + (p.max_q > 1 ? row0 / p.group : 0) + 1;
      const int max_pos = r.L - r.n + (p.max_q > 1 ? (row0 + rows - 1) / p.group : 0);
      const int max_lo = p.window > 0 ? max_pos + 1 - p.window : 0;

      float o[NT][KS][4];
      float m0[NT], m1[NT], l0[NT], l1[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        m0[j] = m1[j] = -INFINITY;
        l0[j] = l1[j] = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[j][i][k] = 0.f;
      }

      const int it0 = it;  // of the part's first tile
      for (int x = kGroups ? x0 : x0 + ((wi - it0) & (GW - 1)); x < x1; x += kGroups ? 1 : GW) {
        it = it0 + (x - x0);
        const int st = it % S;
        if constexpr (kGroups) {  // another warp's tile: its slot is released by all warps
          if (it % GW != wi) {
            if (issued(it) && lane == 0) mbar_arrive(smem_u32(&bar_empty[st]));
            continue;
          }
        }
        // A parity wait is only unambiguous against the phase in progress. The slot's previous
        // tile may be another warp's (GW need not divide S) and copies may land out of
        // order, so the tile must have been issued first: that tells that the slot's earlier
        // phases are complete.
        if (!issued(it) ||
            !warp_wait(smem_u32(&bar_full[st]), (it / S) & 1, abort_flag, p.dev_status))
          continue;  // the run is lost; the barriers below still need every warp
        const int tile0 = (x < r.st ? x : r.lt + x - r.st) * TK;
        const uint32_t sk = ring + st * C::kStageBytes, sv = sk + C::kKBytes;
        const uint32_t okp = s_meta[st].ok;
        const bool all_pieces = okp == (1u << n_pieces) - 1u;
        if (okp != 0 && rows > 0) {
          // ---- values of keys nobody sees must not meet a weight of zero as NaN
          if (!(all_pieces && tile0 + TK <= r.L && (tile0 >= r.lo || tile0 + TK <= r.sinks))) {
            for (int row = lane / 4; row < TK; row += 8) {
              const int key = tile0 + row;
              const bool seen = ((okp >> ((row >> 4) >> piece_shift)) & 1u) && key < r.L &&
                                (key >= r.lo || key < r.sinks);
              if (!seen)
                for (int c = lane & 3; c < C::kRowBytes / 16; c += 4) {
                  const uint32_t at = chunk_at<TK, C::kPanelBytes>(sv, row, c);
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0)
                               : "memory");
                }
            }
            fence_proxy_async_smem();  // before the slot is handed back to TMA
            __syncwarp();
          }
#pragma unroll 1
          for (int pass = 0; pass < C::kMT / MT; ++pass) {
            const int mt0 = pass * MT, key0 = tile0 + mt0 * 16;  // m tiles [mt0, mt0 + MT)
            // ---- S^T = K Q^T
            float s[NT][MT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[j][mt][k] = 0.f;
            // 16-byte chunks of the rows outside: a chunk's q fragments serve all m tiles
            constexpr int kChunks = F8 ? D / 64 : D / 32;  // chunks per lane and row
            constexpr int kSteps = F8 ? 4 : 2;             // k steps of a chunk
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              // e4m3: chunk c of this lane's D/64; bf16: panel c / 2, chunk 2 t4 + c % 2
              const int ch = F8 ? (D / 64) * t4 + c : (c / 2) * 8 + 2 * t4 + (c & 1);
              uint32_t bq[NT][kSteps / 2][4];
#pragma unroll
              for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int h = 0; h < kSteps / 2; ++h) q_frag(j, c * kSteps + 2 * h, bq[j][h]);
              // two m tiles at a time, their products in turn: a product's accumulator is ready
              // again 2 NT products later
#pragma unroll
              for (int m0t = 0; m0t < MT; m0t += 2) {
                uint32_t wa[2][4], wb[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const int row = (mt0 + m0t + u) * 16 + g8;
                  const uint4 va = lds128(chunk_at<TK, C::kPanelBytes>(sk, row, ch));
                  const uint4 vb = lds128(chunk_at<TK, C::kPanelBytes>(sk, row + 8, ch));
                  wa[u][0] = va.x;
                  wa[u][1] = va.y;
                  wa[u][2] = va.z;
                  wa[u][3] = va.w;
                  wb[u][0] = vb.x;
                  wb[u][1] = vb.y;
                  wb[u][2] = vb.z;
                  wb[u][3] = vb.w;
                }
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    uint32_t af[4];
                    if constexpr (F8) {
                      af[0] = e4m3_lo(wa[u][k]);
                      af[1] = e4m3_lo(wb[u][k]);
                      af[2] = e4m3_hi(wa[u][k]);
                      af[3] = e4m3_hi(wb[u][k]);
                    } else {
                      af[0] = wa[u][2 * k];
                      af[1] = wb[u][2 * k];
                      af[2] = wa[u][2 * k + 1];
                      af[3] = wb[u][2 * k + 1];
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                      mma16<F8>(s[j][m0t + u], af, bq[j][k / 2][2 * (k & 1)],
                                bq[j][k / 2][2 * (k & 1) + 1]);
                  }
              }
            }
            // ---- scores in the exp2 domain, masks, running reference
            const bool clear = all_pieces && key0 + MT * 16 <= min_end &&
                               (p.window == 0 || key0 >= max_lo || key0 + MT * 16 <= p.sinks);
            float t0m[NT], t1m[NT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float ks = 1.f, vl = 0.f;
              if constexpr (F8) {
                ks = s_meta[st].ks[(mt0 + mt) >> piece_shift];
                vl = s_meta[st].vl[(mt0 + mt) >> piece_shift];
              }
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                const float a0 = f0[j] * ks, a1 = f1[j] * ks;
                float(&v)[4] = s[j][mt];
                v[0] = fmaf(v[0], a0, vl);
                v[1] = fmaf(v[1], a1, vl);
                v[2] = fmaf(v[2], a0, vl);
                v[3] = fmaf(v[3], a1, vl);
              }
            }
            if (!clear) {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                const bool here = (okp >> ((mt0 + mt) >> piece_shift)) & 1u;
                const int ka = key0 + mt * 16 + g8, kb = ka + 8;
                auto sees = [&](int key, int pos) {
                  return here && key <= pos &&
                         (p.window == 0 || key > pos - p.window || key < p.sinks);
                };
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                  float(&v)[4] = s[j][mt];
                  if (!sees(ka, pos0[j])) v[0] = -INFINITY;
                  if (!sees(ka, pos1[j])) v[1] = -INFINITY;
                  if (!sees(kb, pos0[j])) v[2] = -INFINITY;
                  if (!sees(kb, pos1[j])) v[3] = -INFINITY;
                }
              }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              t0m[j] = t1m[j] = -INFINITY;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                t0m[j] = fmax3(t0m[j], s[j][mt][0], s[j][mt][2]);
                t1m[j] = fmax3(t1m[j], s[j][mt][1], s[j][mt][3]);
              }
            }
            bool move = false;
#pragma unroll
            for (int j = 0; j < NT; ++j)
              move = move || t0m[j] > m0[j] + kThr || t1m[j] > m1[j] + kThr;
            if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
              for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                  t0m[j] = fmaxf(t0m[j], __shfl_xor_sync(0xFFFFFFFFu, t0m[j], d));
                  t1m[j] = fmaxf(t1m[j], __shfl_xor_sync(0xFFFFFFFFu, t1m[j], d));
                }
                const float n0 = fmaxf(m0[j], t0m[j]), n1 = fmaxf(m1[j], t1m[j]);
                const float al0 = n0 == -INFINITY ? 1.f : ex2_approx(m0[j] - n0);
                const float al1 = n1 == -INFINITY ? 1.f : ex2_approx(m1[j] - n1);
                m0[j] = n0;
                m1[j] = n1;
                l0[j] *= al0;
                l1[j] *= al1;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                  o[j][i][0] *= al0;
                  o[j][i][1] *= al1;
                  o[j][i][2] *= al0;
                  o[j][i][3] *= al1;
                }
              }
            }
            // ---- P and O^T += V^T P^T
            float e0[NT], e1[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              e0[j] = m0[j] == -INFINITY ? 0.f : m0[j] - kBias;
              e1[j] = m1[j] == -INFINITY ? 0.f : m1[j] - kBias;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float vi = 1.f;
              if constexpr (F8) vi = s_meta[st].vi[(mt0 + mt) >> piece_shift];
              uint32_t b0[NT], b1[NT];
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                float pr[4];
                pr[0] = ex2_approx(s[j][mt][0] - e0[j]);
                pr[1] = ex2_approx(s[j][mt][1] - e1[j]);
                pr[2] = ex2_approx(s[j][mt][2] - e0[j]);
                pr[3] = ex2_approx(s[j][mt][3] - e1[j]);
                l0[j] = fmaf(pr[0] + pr[2], vi, l0[j]);
                l1[j] = fmaf(pr[1] + pr[3], vi, l1[j]);
                b0[j] = movm(F8 ? pack_f16x2(pr[0], pr[1]) : pack_bf16x2(pr[0], pr[1]));
                b1[j] = movm(F8 ? pack_f16x2(pr[2], pr[3]) : pack_bf16x2(pr[2], pr[3]));
              }
              if constexpr (F8) {
                // words of rows 2t, 2t + 1, 2t + 8, 2t + 9; d = (D/8) g8 + ...
                constexpr int kWords = D / 32;  // 4-byte words per lane and row
                uint32_t w[4][kWords];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int row = (mt0 + mt) * 16 + 2 * t4 + (k & 1) + (k >> 1) * 8;
                  if constexpr (kWords == 4) {
                    const uint4 v = lds128(chunk_at<TK, C::kPanelBytes>(sv, row, g8));
                    w[k][0] = v.x;
                    w[k][1] = v.y;
                    w[k][2] = v.z;
                    w[k][3] = v.w;
                  } else {
                    const uint2 v =
                        lds64(chunk_at<TK, C::kPanelBytes>(sv, row, g8 >> 1) + (g8 & 1) * 8);
                    w[k][0] = v.x;
                    w[k][1] = v.y;
                  }
                }
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                  const uint32_t xa = __byte_perm(w[0][i], w[1][i], 0x5140),
                                 xb = __byte_perm(w[0][i], w[1][i], 0x7362),
                                 ya = __byte_perm(w[2][i], w[3][i], 0x5140),
                                 yb = __byte_perm(w[2][i], w[3][i], 0x7362);
                  const uint32_t a0[4] = {e4m3_lo(xa), e4m3_hi(xa), e4m3_lo(ya), e4m3_hi(ya)};
                  const uint32_t a1[4] = {e4m3_lo(xb), e4m3_hi(xb), e4m3_lo(yb), e4m3_hi(yb)};
#pragma unroll
                  for (int j = 0; j < NT; ++j) {
                    mma16<F8>(o[j][2 * i], a0, b0[j], b1[j]);
                    mma16<F8>(o[j][2 * i + 1], a1, b0[j], b1[j]);
                  }
                }
              } else {
                const int row = (mt0 + mt) * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                  uint32_t a[4];
                  ldsm_x4_trans(a, chunk_at<TK, C::kPanelBytes>(sv, row, 2 * i + ((lane >> 3) & 1)));
#pragma unroll
                  for (int j = 0; j < NT; ++j) mma16<F8>(o[j][i], a, b0[j], b1[j]);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_empty[st]));
      }

      it = it0 + (x1 - x0);
      // ---- join the row group's warps: the largest reference first, then warp wi sums m tiles
      // [wi MQ, (wi + 1) MQ) of all of them
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l0[j] += __shfl_xor_sync(0xFFFFFFFFu, l0[j], d);
          l1[j] += __shfl_xor_sync(0xFFFFFFFFu, l1[j], d);
        }
        if (g8 == 0)
          *reinterpret_cast<float2*>(&s_m[warp][j * 8 + 2 * t4]) = make_float2(m0[j], m1[j]);
      }
      group_sync();
      float top0[NT], top1[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        top0[j] = top1[j] = -INFINITY;
#pragma unroll
        for (int w = 0; w < GW; ++w) {
          const float2 m = *reinterpret_cast<const float2*>(&s_m[rg * GW + w][j * 8 + 2 * t4]);
          top0[j] = fmaxf(top0[j], m.x);
          top1[j] = fmaxf(top1[j], m.y);
        }
        const float a0 = m0[j] == -INFINITY ? 0.f : ex2_approx(m0[j] - top0[j]);
        const float a1 = m1[j] == -INFINITY ? 0.f : ex2_approx(m1[j] - top1[j]);
        if (g8 == 0)
          *reinterpret_cast<float2*>(&s_l[warp][j * 8 + 2 * t4]) = make_float2(l0[j] * a0, l1[j] * a1);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          o[j][i][0] *= a0;
          o[j][i][1] *= a1;
          o[j][i][2] *= a0;
          o[j][i][3] *= a1;
        }
      }
      // slot of (summing warp, source warp) of the group: every source but itself
      constexpr int kSlot = NT * MQ * 4 * 32;
      float* const group_join = join + rg * (GW * (GW - 1) * kSlot) + lane;
#pragma unroll
      for (int dst = 0; dst < GW; ++dst) {
        if (dst == wi) continue;
        float* to = group_join + (dst * (GW - 1) + (wi < dst ? wi : wi - 1)) * kSlot;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < MQ; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              to[((j * MQ + i) * 4 + k) * 32] = o[j][dst * MQ + i][k];
      }
      group_sync();
      const bool final = whole_l && whole_r;
      float* part = p.parts + (size_t)(2 * blockIdx.x + (whole_l ? 1 : 0)) * (p.unit_rows * (D + 2));
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float acc[MQ][4];
#pragma unroll
        for (int d = 0; d < GW; ++d)
          if (d == wi) {
#pragma unroll
            for (int i = 0; i < MQ; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[i][k] = o[j][d * MQ + i][k];
          }
        // ((own + first) + second) + third other: the same order every time
#pragma unroll
        for (int w = 0; w < GW - 1; ++w) {
          const float* from = group_join + (wi * (GW - 1) + w) * kSlot;
#pragma unroll
          for (int i = 0; i < MQ; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][k] += from[((j * MQ + i) * 4 + k) * 32];
        }
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < GW; ++w) {
          const float2 l = *reinterpret_cast<const float2*>(&s_l[rg * GW + w][j * 8 + 2 * t4]);
          sum.x += l.x;
          sum.y += l.y;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // column 2 t4 + k: one q row
          const int row = j * 8 + 2 * t4 + k;
          const float l = k ? sum.y : sum.x, top = k ? top1[j] : top0[j];
          const float inv = !final ? 1.f : l > 0.f ? 1.f / l : 0.f;
          float v[2 * MQ];
#pragma unroll
          for (int i = 0; i < MQ; ++i) {
            v[2 * i] = acc[i][k] * inv;
            v[2 * i + 1] = acc[i][k + 2] * inv;
          }
          int64_t at = 0;
          if (row >= rows) continue;
          if (final) {
            const int rr = row0 + row, tok = p.max_q > 1 ? rr / p.group : 0;
            at = (int64_t)(r.q0 + tok) * p.hq + g * p.group + (rr - tok * p.group);
          }
          float* to32 = final ? static_cast<float*>(p.out) + at * D : part + (rg * GR + row) * D;
          uint16_t* to16 = static_cast<uint16_t*>(p.out) + at * D;
          const bool half = final && p.out_bf16;
          if constexpr (F8) {  // elements d0 .. d0 + 2 MQ - 1 of the row
            const int d0 = (D / 8) * g8 + 2 * MQ * wi;
            if constexpr (MQ >= 2) {
#pragma unroll
              for (int i = 0; i < 2 * MQ; i += 4) {
                if (half)
                  *reinterpret_cast<uint2*>(to16 + d0 + i) =
                      make_uint2(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]));
                else
                  *reinterpret_cast<float4*>(to32 + d0 + i) =
                      make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
              }
            } else {
              if (half)
                *reinterpret_cast<uint32_t*>(to16 + d0) = pack_bf16x2(v[0], v[1]);
              else
                *reinterpret_cast<float2*>(to32 + d0) = make_float2(v[0], v[1]);
            }
          } else {  // elements 16 m + g8 and 16 m + g8 + 8 of m tile m
#pragma unroll
            for (int i = 0; i < 2 * MQ; ++i) {
              const int d = 16 * (wi * MQ + i / 2) + g8 + 8 * (i & 1);
              if (half)
                to16[d] = (uint16_t)pack_bf16x2(v[i], 0.f);
              else
                to32[d] = v[i];
            }
          }
          if (wi == 0 && g8 == 0) {
            if (final) {
              if (p.lse != nullptr)
                p.lse[at] = l > 0.f ? (top - kBias + log2f(l)) * kLn2 : -INFINITY;
            } else {
              *reinterpret_cast<float2*>(part + p.unit_rows * D + 2 * (rg * GR + row)) = make_float2(top, l);
            }
          }
        }
      }
      if (!whole_l && whole_r && tid == 0) {
        // the unit ends here: tell the second launch where it began
        const int begin = before - x0;  // list place of the unit's first tile
        const int longer = more * (len + 1);  // tiles of the runs with one more
        const int c0 = begin < longer
                           ? (int)((unsigned)begin / (unsigned)(len + 1))
                           : more + (int)((unsigned)(begin - longer) / (unsigned)len);
        p.jobs[blockIdx.x] = make_int4(c0, min(r.n * p.group - rt * p.unit_rows, p.unit_rows),
                                        rt * p.unit_rows, g);
        p.job_q0[blockIdx.x] = r.q0;
      }
      group_sync();  // before the next unit's references and sums
    };
    [[maybe_unused]] int last = 0;  // row groups of the part before
    while (left > 0) {
      int g, rt, x0, x1;
      const int before = t1 - left;
      if (!next_seg(g, rt, x0, x1)) continue;
      const int rows = kGroups ? min(r.n * p.group - rt * p.unit_rows, p.unit_rows) : 0;
      if constexpr (kGroups) {
        // Groups of another size lay their q rows and accumulators over one another's: all warps
        // must be done with the part before (each group waits only for its own warps there).
        const int groups = rows > 2 * GR ? 4 : rows > GR ? 2 : 1;
        if (last != 0 && groups != last) named_barrier_sync(1, kNW * 32);
        last = groups;
      }
      if (rows > 2 * GR)
        segment(std::integral_constant<int, kGroups ? 4 : 1>(), g, rt, x0, x1, before);
      else if (rows > GR)
        segment(std::integral_constant<int, kGroups ? 2 : 1>(), g, rt, x0, x1, before);
      else
        segment(std::integral_constant<int, 1>(), g, rt, x0, x1, before);
    }
  }
}

// Joins the parts of the units that CTA borders cut: block (c, y) for rows y, y + kJoinRows, ..
// of the unit that ended in CTA c (with a block for each of 64 rows most blocks are empty: 4
// requests x 3000 keys, 40 rows 25 -> 20 us). Four warps take every fourth part each, kBatch
// parts' loads in flight (a unit of one long request may have hundreds), then the warps'
// results are joined in order.
constexpr int kJoinRows = 16;
template <int D, bool kMany>  // kMany: more rows than that
__global__ void __launch_bounds__(128) attn_decode_join_kernel(const Params p, float bias) {
  constexpr int kWarps = 4, kBatch = 4;
  const int R = p.unit_rows;
  __shared__ float2 s_ml[kWarps];
  __shared__ float4 s_acc[kWarps][D / 4];
  const int c1 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_prior_grids();  // the parts are written
  const int4 job = p.jobs[c1];
  const int q0 = p.job_q0[c1];
  if (job.x < 0 || (int)blockIdx.y >= job.y) return;
  const bool mine = lane < D / 4;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int row = blockIdx.y; row < job.y; row += kJoinRows) {
    float top = -INFINITY, sum = 0.f;
    float4 acc = zero;
    for (int c = job.x + warp; c <= c1; c += kWarps * kBatch) {
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int cc = c + i * kWarps;
        ml[i] = make_float2(-INFINITY, 0.f);
        v[i] = zero;
        if (cc <= c1) {
          const float* part = p.parts + (size_t)(2 * cc + (cc == job.x ? 1 : 0)) * (R * (D + 2));
          ml[i] = *reinterpret_cast<const float2*>(part + R * D + 2 * row);
          if (mine) v[i] = *reinterpret_cast<const float4*>(part + row * D + lane * 4);
        }
      }
      float n = top;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) n = fmaxf(n, ml[i].x);
      const float f = top == -INFINITY ? 0.f : ex2_approx(top - n);
      top = n;
      sum *= f;
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float fi = ml[i].x == -INFINITY ? 0.f : ex2_approx(ml[i].x - n);
        sum = fmaf(ml[i].y, fi, sum);
        acc.x = fmaf(v[i].x, fi, acc.x);
        acc.y = fmaf(v[i].y, fi, acc.y);
        acc.z = fmaf(v[i].z, fi, acc.z);
        acc.w = fmaf(v[i].w, fi, acc.w);
      }
    }
    if (lane == 0) s_ml[warp] = make_float2(top, sum);
    if (mine) s_acc[warp][lane] = acc;
    __syncthreads();
    if (warp == 0) {
      float m = -INFINITY, l = 0.f;
      float4 o = zero;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_ml[w].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w];
        const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
        l = fmaf(ml.y, f, l);
        if (mine) {
          const float4 v = s_acc[w][lane];
          o.x = fmaf(v.x, f, o.x);
          o.y = fmaf(v.y, f, o.y);
          o.z = fmaf(v.z, f, o.z);
          o.w = fmaf(v.w, f, o.w);
        }
      }
      const int rr = job.z + row, tok = rr / p.group;
      const int64_t at = (int64_t)(q0 + tok) * p.hq + job.w * p.group + (rr - tok * p.group);
      const float inv = l > 0.f ? 1.f / l : 0.f;
      if (mine) {
        if (p.out_bf16) {
          uint2* to = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at * D) + lane;
          *to = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        } else {
          reinterpret_cast<float4*>(static_cast<float*>(p.out) + at * D)[lane] =
              make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        }
      }
      if (p.lse != nullptr && lane == 0)
        p.lse[at] = l > 0.f ? (m - bias + log2f(l)) * kLn2 : -INFINITY;
    }
    if (!kMany) return;
    if (row + kJoinRows < job.y) __syncthreads();  // before the next row's results
  }
}

// Rows of a unit: the least of 8, 16, 32 and 64 that holds a request's rows of one KV head (64
// for more, in several units).
int rows_of(int max_q, int group) {
  const int64_t rows = (int64_t)max_q * group;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}
size_t job_bytes(size_t ctas) {
  return (ctas * (sizeof(int4) + sizeof(int)) + 255) / 256 * 256;
}

template <bool F8, int D, int NT, bool kGroups>
cudaError_t launch(const AttnDecodeArgs& a, int dev, int sms, int* drv_err, cudaStream_t stream) {
  using C = Cfg<F8, D, NT>;
  Params p;
  p.q = static_cast<const uint16_t*>(a.q);
  p.cu_q = a.cu_q;
  p.page_tables = a.page_tables;
  p.kv_lens = a.kv_lens;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.out = a.out;
  p.lse = a.lse;
  p.dev_status = a.dev_status;
  p.total_q = (int)a.total_q;
  p.max_keys = a.max_pages * a.page_size;
  p.batch = a.batch;
  p.max_q = a.max_q;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.group = a.hq / a.hkv;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.page_size = a.page_size;
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.page_size) ++p.page_shift;
  p.window = a.window;
  p.sinks = a.sinks;
  p.scale_log2 = a.scale * kLog2e;
  p.out_bf16 = a.out_bf16 ? 1 : 0;
  p.ctas = kCtasPerSm * sms;
  p.unit_rows = rows_of(a.max_q, p.group);
  p.row_shift = 0;
  while ((1 << p.row_shift) < p.unit_rows) ++p.row_shift;
  p.jobs = static_cast<int4*>(a.workspace);
  p.job_q0 = reinterpret_cast<int*>(p.jobs + p.ctas);
  p.parts =
      reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + job_bytes((size_t)p.ctas));
  CUtensorMap mk, mv;
  auto make = [&](CUtensorMap* m, void* base) -> bool {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.page_size, (uint64_t)a.num_pages * a.hkv};
    const uint64_t strides[2] = {(uint64_t)C::kRowBytes, (uint64_t)C::kRowBytes * a.page_size};
    const uint32_t box[3] = {(uint32_t)(F8 ? D : 64),
                             (uint32_t)(a.page_size < C::kTK ? a.page_size : C::kTK), 1};
    const CUresult e = encode_tensor_map(
        m, F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims,
        strides, box, C::kPanelBytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
    if (e != CUDA_SUCCESS) *drv_err = (int)e;
    return e == CUDA_SUCCESS;
  };
  if (!make(&mk, const_cast<void*>(a.k_cache)) || !make(&mv, const_cast<void*>(a.v_cache)))
    return cudaErrorInvalidValue;
  // The kernel's shared-memory limit is set once per device (bit i: device i), not per call: 0.8 of
  // the 9 us that a small call takes the host. A launch that fails has it set again.
  static std::atomic<uint64_t> set{0};
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  cudaError_t e = cudaSuccess;
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(attn_decode_kernel<F8, D, NT, kGroups>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  e = launch_ahead(attn_decode_kernel<F8, D, NT, kGroups>, dim3(p.ctas), kThreads, C::kSmemBytes,
                   stream, mk, mv, p);
  if (e != cudaSuccess) {
    set.fetch_and(~bit, std::memory_order_relaxed);
    return e;
  }
  const bool many = p.unit_rows > kJoinRows;
  return launch_ahead(many ? attn_decode_join_kernel<D, true> : attn_decode_join_kernel<D, false>,
                      dim3(p.ctas, many ? kJoinRows : p.unit_rows), 128, 0, stream, p,
                      F8 ? 11.f : 0.f);
}

template <bool F8, int D>
cudaError_t launch_nt(const AttnDecodeArgs& a, int dev, int sms, int* drv_err,
                      cudaStream_t stream) {
  switch (rows_of(a.max_q, a.hq / a.hkv)) {
    case 8: return launch<F8, D, 1, false>(a, dev, sms, drv_err, stream);
    case 16: return launch<F8, D, 2, false>(a, dev, sms, drv_err, stream);
    default: return launch<F8, D, 2, true>(a, dev, sms, drv_err, stream);
  }
}

}  // namespace

size_t attn_decode_workspace_bytes(int max_q, int hq, int hkv, int d, int sms) {
  const size_t ctas = (size_t)kCtasPerSm * sms, rows = rows_of(max_q, hq / hkv);
  return job_bytes(ctas) + ctas * 2 * rows * (d + 2) * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, int* drv_err, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (a.d == 64)
    return a.f8 ? launch_nt<true, 64>(a, dev, sms, drv_err, stream)
                : launch_nt<false, 64>(a, dev, sms, drv_err, stream);
  if (a.d == 128)
    return a.f8 ? launch_nt<true, 128>(a, dev, sms, drv_err, stream)
                : launch_nt<false, 128>(a, dev, sms, drv_err, stream);
  return cudaErrorInvalidValue;
}

}  // namespace tts
