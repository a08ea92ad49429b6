// Append of new tokens to a paged grouped-query KV cache, the position rotation applied on
// the way: q and k of every new token are rotated (rotate-half pairs (j, j + d/2), the
// cos/sin table of tts_rope_cache, as in tts_qkv_rope), q goes to q_out, k and v to their
// page as bf16 or as e4m3 codes with one power-of-two scale per (page, KV head).
//
// The e4m3 scale of a page and head is the smallest power of two s (at least 2^-60) with
// |x| <= 448 s for every row the page holds. A page begun by the call takes it from the new
// rows alone; a page that already holds rows keeps the larger of its scale and the new
// rows', and when it grows the earlier rows' codes are divided by the ratio. With powers of
// two that move rounds nothing except where a code falls below 2^-6 (e4m3's subnormals), so
// appending token by token loses nothing over quantizing the page at once; the price, up to
// one binade of e4m3's eighteen, costs no mantissa bit.
//
// Bound: HBM. A prompt token moves (4 Hq + (6 + 2 c) Hkv) d bytes (c = 2 or 1 bytes per cached
// value; k_out included), read and written once: a page of one head stays in registers between
// the maximum and the rounding, and the rotation's table row is read once per eight q heads.
// 36,411 tokens of 32 / 8 heads of 128 into e4m3: 147 us, 6.1 TB/s, 0.90 of the measured copy
// rate (what is left: the blocks' chain of lengths, rows, reduction and stores, 50 % of the warps
// resident). A step is one launch's latency: 3.0 us for 8 requests, 3.3 for 64. Where a page grows
// its scale one warp reads and rewrites the page's earlier rows: 64 requests whose k and v pages
// all grow take 6.1 us at slot 60 of pages of 64, 8.1 at slot 120 of 128.
//
// kAxes: positions are the caller's, on up to four axes, and two bits per rotation pair choose the
// one whose table row it takes; eight pairs of one axis are loaded as without axes. The price is a
// load in front of the table's: 26,800 prompt tokens with three axes into e4m3 118 us, 0.82 of the copy
// rate; 16 trees of 25 to 64 tokens into bf16 7.2 us, one wave of blocks.
#include <cstdint>
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tts {
namespace {

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint2 quant8(const float* f, float inv) {
  return make_uint2(cvt_e4m3x2(f[0] * inv, f[1] * inv) | (cvt_e4m3x2(f[2] * inv, f[3] * inv) << 16),
                    cvt_e4m3x2(f[4] * inv, f[5] * inv) | (cvt_e4m3x2(f[6] * inv, f[7] * inv) << 16));
}

// cos / sin of the 8 pairs [8c, 8c + 8) at one position.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(const float* __restrict__ cs, Turn& t) {
  const float4* p = reinterpret_cast<const float4*>(cs);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(p + i);
    t.c[2 * i] = v.x;
    t.s[2 * i] = v.y;
    t.c[2 * i + 1] = v.z;
    t.s[2 * i + 1] = v.w;
  }
}
// The same with explicit positions: pair j turns by the table's row at the token's position on axis
// pair_axis[j] (two bits a pair). False, and no turn, where a position lies outside the table.
struct Positions {
  int at[4];
};
__device__ __forceinline__ void load_positions(const KvAppendArgs& p, int64_t tok, Positions& pos) {
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    pos.at[a] = 0;
    if (a < p.axes) pos.at[a] = __ldg(p.positions + a * p.total_new + tok);
  }
}
template <int D>
__device__ __forceinline__ bool load_turn_axes(const KvAppendArgs& p, const Positions& from, int c,
                                               Turn& t) {
  const int(&pos)[4] = from.at;
  bool ok = true;
#pragma unroll
  for (int a = 0; a < 4; ++a) ok = ok && pos[a] >= 0 && pos[a] < p.max_pos;
  const uint32_t axis = (uint32_t)(p.pair_axis[c >> 2] >> ((c & 3) * 16)) & 0xFFFFu;
  auto row = [&](uint32_t a) -> const float* {  // pairs [8c, 8c + 8) at the position on axis a
    const int at = !ok ? 0 : a & 2 ? (a & 1 ? pos[3] : pos[2]) : (a & 1 ? pos[1] : pos[0]);
    return p.cos_sin + ((int64_t)at * (D / 2) + c * 8) * 2;
  };
  if (axis == (axis & 3) * 0x5555u) {
    load_turn(row(axis & 3), t);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = __ldg(reinterpret_cast<const float2*>(row((axis >> (2 * i)) & 3)) + i);
      t.c[i] = v.x;
      t.s[i] = v.y;
    }
  }
  return ok;
}
// The rotation, every product and sum rounded on its own (no contraction: the result does
// not depend on which of two products an FMA would keep exact).
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const Turn& t) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __fsub_rn(__fmul_rn(a[i], t.c[i]), __fmul_rn(b[i], t.s[i]));
    b[i] = __fadd_rn(__fmul_rn(a[i], t.s[i]), __fmul_rn(b[i], t.c[i]));
    a[i] = x;
  }
}

struct Req {
  int64_t t0;  // first new token's row
  int n;       // new tokens (0: nothing to do)
  int past;    // tokens already in the cache
  bool ok;     // positions fit the page table and the cos/sin table
};
template <bool kAxes>
__device__ __forceinline__ Req make_req(const KvAppendArgs& p, int a, int e, int past,
                                        uint32_t* bad) {
  Req r;
  r.t0 = a;
  r.n = 0;
  r.past = past;
  r.ok = false;
  if (a < 0 || e < a || e > p.total_new || e - a > p.max_new) {
    *bad |= kDevBadArg;
    return r;
  }
  r.n = e - a;
  const int64_t end = (int64_t)past + r.n;
  r.ok = past >= 0 && end <= ((int64_t)p.max_pages << p.page_shift) &&
         (kAxes || p.cos_sin == nullptr || end <= p.max_pos);
  if (!r.ok && r.n > 0) *bad |= kDevIndexRange;
  return r;
}
template <bool kAxes>
__device__ __forceinline__ Req load_req(const KvAppendArgs& p, int b, uint32_t* bad) {
  return make_req<kAxes>(p, p.cu_new[b], p.cu_new[b + 1], p.past_lens[b], bad);
}

// The request that owns unit u, where request b owns units [cu[b] / size + 2b, cu[b+1] / size +
// 2(b+1)): at least as many as it has pieces of `size` = 2^shift tokens, whatever their offset.
// Warp-collective: the last b whose first unit is <= u, found 32 bounds at a time; with up to 32
// requests the one round of loads brings the request itself too.
template <bool kAxes>
__device__ __forceinline__ Req find_request(const KvAppendArgs& p, int shift, int64_t u, int* b,
                                            int64_t* first) {
  const int lane = threadIdx.x & 31;
  uint32_t bad = 0;
  if (p.batch <= 32) {
    int a = 0, e = 0, past = 0;
    if (lane < p.batch) {
      a = p.cu_new[lane];
      e = p.cu_new[lane + 1];
      past = p.past_lens[lane];
    }
    const int64_t begin = (int64_t)(a >> shift) + 2 * lane;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, lane < p.batch && begin <= u);
    *b = m ? 31 - __clz(m) : 0;
    *first = __shfl_sync(0xFFFFFFFFu, begin, *b);
    return make_req<kAxes>(p, __shfl_sync(0xFFFFFFFFu, a, *b), __shfl_sync(0xFFFFFFFFu, e, *b),
                    __shfl_sync(0xFFFFFFFFu, past, *b), &bad);
  }
  int lo = 0, span = p.batch;
  while (true) {
    const int step = (span + 31) >> 5;
    const int i = lo + lane * step;
    const bool below =
        i < p.batch && i < lo + span && (int64_t)(p.cu_new[i] >> shift) + 2 * i <= u;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, below);
    const int last = m ? 31 - __clz(m) : 0;
    span = min(step, span - last * step);
    lo += last * step;
    if (step == 1) break;
  }
  *b = lo;
  *first = (int64_t)(p.cu_new[lo] >> shift) + 2 * lo;
  return load_req<kAxes>(p, lo, &bad);
}

// Report bad requests once (block 0 of either kernel).
template <bool kAxes>
__device__ __forceinline__ void report(const KvAppendArgs& p) {
  if (p.dev_status == nullptr) return;
  uint32_t bad = 0;
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) load_req<kAxes>(p, b, &bad);
  if (bad) atomicOr(p.dev_status, bad);
}

// ---- one page of one head ----------------------------------------------------------------
// Rows [f, f + nr) of the request's pi-th touched page, head g, held by `lanes` threads: thread
// `id` holds, per pass, 16 values of row id / (D/16): [8c, 8c + 8) and the same of the row's
// second half, c = id % (D/16), i.e. both members of eight rotation pairs. kWarp: the threads
// are one warp; else they are the block, and all of it comes here together.
template <int D, bool kF8, int kPasses, bool kWarp, bool kAxes>
__device__ __forceinline__ void append_page(const KvAppendArgs& p, int b, const Req& r, int pi,
                                            int g, bool is_v, int id, int lanes, float* s_red) {
  constexpr int kTpr = D / 16;  // threads per row
  const int ps = 1 << p.page_shift;
  if (r.n <= 0) return;
  // A past that fails r.ok caches nothing; its k_out rows are walked from position 0. Positions
  // that pass are below 2^30.
  const int past = r.ok ? r.past : 0;
  const int page_log = (past >> p.page_shift) + pi, first_pos = page_log << p.page_shift;
  const int lo = max(past, first_pos), hi = min(past + r.n, first_pos + ps);
  if (pi > (r.n >> p.page_shift) + 1 || lo >= hi) return;
  const int f = lo - first_pos, nr = hi - lo;
  const int64_t tok0 = r.t0 + (lo - past);
  // The new rows are asked for before the page: a block that waited for the one and then the
  // other kept too little in flight (36,000 prompt tokens 167 -> 158 us).
  const int c = id % kTpr, row_in = id / kTpr, rows_per = lanes / kTpr;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.v : p.k) + (int64_t)g * D + c * 8;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  uint4 raw[kPasses][2];
  [[maybe_unused]] Positions pos[kAxes ? kPasses : 1];
#pragma unroll
  for (int s = 0; s < kPasses; ++s) {
    const int row = s * rows_per + row_in;
    if constexpr (kAxes) {
      if (!is_v && row < nr) load_positions(p, tok0 + row, pos[s]);
    }
    raw[s][0] = raw[s][1] = make_uint4(0, 0, 0, 0);
    if (row < nr) {
      const uint16_t* at = src + (tok0 + row) * stride;
      raw[s][0] = *reinterpret_cast<const uint4*>(at);
      raw[s][1] = *reinterpret_cast<const uint4*>(at + D / 2);
    }
  }
  int64_t pg = -1;
  if (r.ok) {
    pg = p.page_tables[(int64_t)b * p.max_pages + page_log];
    if (pg < 0 || pg >= p.num_pages) {
      pg = -1;
      if (id == 0 && p.dev_status != nullptr) atomicOr(p.dev_status, kDevIndexRange);
    }
  }
  const bool want_k = !is_v && p.k_out != nullptr;
  if (pg < 0 && !want_k) return;
  const int64_t ph = pg * p.hkv + g;  // (page, head) of the cache
  float* scale_at = is_v ? p.v_scale : p.k_scale;
  float old = 0.f;
  if constexpr (kF8) {
    if (pg >= 0 && f > 0) old = scale_at[ph];
  }
  float x[kPasses][16];
  float amax = 0.f;
#pragma unroll
  for (int s = 0; s < kPasses; ++s) {
    const int row = s * rows_per + row_in;
    float(&a)[8] = *reinterpret_cast<float(*)[8]>(&x[s][0]);
    float(&bb)[8] = *reinterpret_cast<float(*)[8]>(&x[s][8]);
    unpack8(raw[s][0], a);
    unpack8(raw[s][1], bb);
    if constexpr (kAxes) {
      if (!is_v && row < nr && r.ok) {
        Turn t;
        if (load_turn_axes<D>(p, pos[s], c, t)) {
          rotate(a, bb, t);
        } else {  // a position outside the table: reported, and the key is zeros
#pragma unroll
          for (int i = 0; i < 16; ++i) x[s][i] = 0.f;
          if (c == 0 && g == 0 && p.dev_status != nullptr) atomicOr(p.dev_status, kDevIndexRange);
        }
      }
    } else if (!is_v && p.cos_sin != nullptr && row < nr && r.ok) {
      Turn t;
      load_turn(p.cos_sin + ((int64_t)(lo + row) * (D / 2) + c * 8) * 2, t);
      rotate(a, bb, t);
    }
    if (want_k && row < nr) {
      uint16_t* o = static_cast<uint16_t*>(p.k_out) + ((tok0 + row) * p.hkv + g) * D + c * 8;
      const uint4 z = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(o) = r.ok ? pack8(a) : z;
      *reinterpret_cast<uint4*>(o + D / 2) = r.ok ? pack8(bb) : z;
    }
    if constexpr (kF8) {
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(x[s][i]));
    }
  }
  if (pg < 0) return;  // the same for every thread of the group
  if constexpr (!kF8) {
    uint16_t* dst = static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache);
#pragma unroll
    for (int s = 0; s < kPasses; ++s) {
      const int row = s * rows_per + row_in;
      if (row < nr) {
        uint16_t* o = dst + (ph * ps + f + row) * D + c * 8;
        *reinterpret_cast<uint4*>(o) = pack8(&x[s][0]);
        *reinterpret_cast<uint4*>(o + D / 2) = pack8(&x[s][8]);
      }
    }
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if constexpr (!kWarp) {
      if ((id & 31) == 0) s_red[id >> 5] = amax;
      __syncthreads();
      for (int w = 0; w < (lanes >> 5); ++w) amax = fmaxf(amax, s_red[w]);
    }
    float sc = block_scale(amax);
    bool fresh = f == 0;
    if (!fresh && !(old > 0.f && old < INFINITY)) {  // no scale a cache row can have
      fresh = true;
      if (id == 0 && p.dev_status != nullptr) atomicOr(p.dev_status, kDevBadArg);
    }
    const bool grow = !fresh && sc > old;
    if (!fresh && !grow) sc = old;
    const float inv = 1.f / sc;
    uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + ph * ps * D;
    if (grow) {  // the page's earlier rows move to the new scale
      const float ratio = old * inv;
      for (int i = id; i < f * (D / 8); i += lanes) {
        uint2* at = reinterpret_cast<uint2*>(dst) + i;
        const uint2 w = *at;
        float y[8];
        const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float2 v = e4m3x2_to_float2((uint16_t)(ww[h >> 1] >> (16 * (h & 1))));
          y[2 * h] = v.x;
          y[2 * h + 1] = v.y;
        }
        *at = quant8(y, ratio);
      }
    }
#pragma unroll
    for (int s = 0; s < kPasses; ++s) {
      const int row = s * rows_per + row_in;
      if (row < nr) {
        uint8_t* o = dst + (int64_t)(f + row) * D + c * 8;
        *reinterpret_cast<uint2*>(o) = quant8(&x[s][0], inv);
        *reinterpret_cast<uint2*>(o + D / 2) = quant8(&x[s][8], inv);
      }
    }
    if (id == 0 && (fresh || grow)) scale_at[ph] = sc;
  }
}

// One row of q by D/16 threads; thread c holds the pairs [8c, 8c + 8).
template <int D>
__device__ __forceinline__ void rotate_q_row(const KvAppendArgs& p, bool ok, int64_t tok, int h,
                                             int c, const Turn& t) {
  const uint16_t* at = static_cast<const uint16_t*>(p.q) + tok * p.q_stride + (int64_t)h * D + c * 8;
  float a[8], b[8];
  unpack8(*reinterpret_cast<const uint4*>(at), a);
  unpack8(*reinterpret_cast<const uint4*>(at + D / 2), b);
  if (p.cos_sin != nullptr) rotate(a, b, t);
  uint16_t* o = static_cast<uint16_t*>(p.q_out) + (tok * p.hq + h) * D + c * 8;
  const uint4 z = make_uint4(0, 0, 0, 0);
  *reinterpret_cast<uint4*>(o) = ok ? pack8(a) : z;
  *reinterpret_cast<uint4*>(o + D / 2) = ok ? pack8(b) : z;
}

constexpr int kQHeads = 8;  // q heads that share one load of the table row

// Prompts: a block per (page, head) of k and of v, and a block per (token tile, 8 q heads).
// Registers are held to 48 (64 for the pages of 2048 pieces), for five (two) blocks per SM: what
// bounds the kernel is how many rows are on their way (28,000 tokens in pages of 128: 75 -> 55 us,
// of 16 to 32: 58 -> 53 us; pages of 64 in blocks of 512 threads instead of 256: 50 -> 64 us), and
// that outweighs what it spills: 20 bytes a thread where a page takes one pass, 44 to 52 where it
// takes two, none at 64 registers. With explicit positions a page of two passes holds two rows' more of
// them: 220 to 250 bytes of spills at 48 registers, none at 64 and four blocks per SM (26,800 prompt tokens
// into e4m3 pages of 64 123 -> 119 us, trees of 25 to 64 tokens 7.9 -> 7.2; pages of one pass 107 -> 112).
template <int D, bool kF8, int kPasses, int kMost, bool kAxes>
__global__ void __launch_bounds__(kMost, kMost == 256 ? (kAxes && kPasses == 2 ? 4 : 5) : 2)
    append_pages_kernel(const KvAppendArgs p, uint64_t q_share, int q_shift, int q_groups) {
  constexpr int kTpr = D / 16;
  __shared__ float s_red[16];
  wait_for_prior_grids();
  if (blockIdx.x == 0) report<kAxes>(p);
  int64_t first;
  // q_share: the part of the blocks that rotates q, as a fraction of 2^32. The two kinds alternate at
  // that rate: what a page's block waits for (its reduction) is filled by a q block's plain
  // streaming (36,000 tokens: 154 us one kind after the other, 147 so).
  const unsigned qb = (unsigned)((blockIdx.x * q_share) >> 32);  // q blocks before this one
  if (qb == (unsigned)(((blockIdx.x + 1ull) * q_share) >> 32)) {
    const unsigned kb = blockIdx.x - qb, heads = 2 * p.hkv;
    const int64_t u = kb / heads;
    const int hh = (int)(kb % heads);
    int b;
    const Req r = find_request<kAxes>(p, p.page_shift, u, &b, &first);
    append_page<D, kF8, kPasses, false, kAxes>(p, b, r, (int)(u - first),
                                               hh >= p.hkv ? hh - p.hkv : hh, hh >= p.hkv,
                                               threadIdx.x, blockDim.x, s_red);
    return;
  }
  const int64_t u = qb / (unsigned)q_groups;
  const int h0 = (int)(qb % (unsigned)q_groups) * kQHeads;
  int b;
  const Req r = find_request<kAxes>(p, q_shift, u, &b, &first);
  const int c = threadIdx.x % kTpr;
  const int64_t i = ((u - first) << q_shift) + threadIdx.x / kTpr;
  if (i < 0 || i >= r.n) return;  // i < 0: units in front of a first bound above 0
  Turn t;
  bool ok = r.ok;
  if constexpr (kAxes) {
    Positions pos;
    load_positions(p, r.t0 + i, pos);
    ok = ok && load_turn_axes<D>(p, pos, c, t);
  } else if (p.cos_sin != nullptr && r.ok) {
    load_turn(p.cos_sin + ((r.past + i) * (D / 2) + c * 8) * 2, t);
  }
  const int h1 = h0 + kQHeads < p.hq ? h0 + kQHeads : p.hq;
#pragma unroll 8
  for (int h = h0; h < h1; ++h) rotate_q_row<D>(p, ok, r.t0 + i, h, c, t);
}

// Steps (a few new tokens per request: all of a page's new rows fit one warp): a warp per
// (request, touched page, head) of k and of v, then D/16 lanes per q row.
template <int D, bool kF8, bool kAxes>
__global__ void __launch_bounds__(128) append_steps_kernel(const KvAppendArgs p, int pages_per,
                                                           int64_t kv_warps) {
  constexpr int kTpr = D / 16;
  wait_for_prior_grids();
  if (blockIdx.x == 0) report<kAxes>(p);
  const int lane = threadIdx.x & 31;
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  uint32_t bad = 0;
  if (w < kv_warps) {
    const int heads = 2 * p.hkv;
    const int hh = (int)(w % heads);
    const int64_t u = w / heads;
    const int b = (int)(u / pages_per);
    const Req r = load_req<kAxes>(p, b, &bad);
    append_page<D, kF8, 1, true, kAxes>(p, b, r, (int)(u % pages_per), hh >= p.hkv ? hh - p.hkv : hh,
                                 hh >= p.hkv, lane, 32, nullptr);
    return;
  }
  if (p.q == nullptr) return;  // the last block's spare warps: there are no q heads to divide by
  const int64_t row = (w - kv_warps) * (32 / kTpr) + lane / kTpr;
  const int h = (int)(row % p.hq);
  const int64_t bi = row / p.hq;
  const int64_t b = bi / p.max_new;
  const int i = (int)(bi % p.max_new);
  if (b >= p.batch) return;
  const Req r = load_req<kAxes>(p, (int)b, &bad);
  if (i >= r.n) return;
  const int c = lane % kTpr;
  Turn t;
  bool ok = r.ok;
  if constexpr (kAxes) {
    Positions pos;
    load_positions(p, r.t0 + i, pos);
    ok = ok && load_turn_axes<D>(p, pos, c, t);
  } else if (p.cos_sin != nullptr && r.ok) {
    load_turn(p.cos_sin + (((int64_t)r.past + i) * (D / 2) + c * 8) * 2, t);
  }
  rotate_q_row<D>(p, ok, r.t0 + i, h, c, t);
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

template <int D, bool kF8, bool kAxes>
cudaError_t launch_append(const KvAppendArgs& p, cudaStream_t stream) {
  constexpr int kTpr = D / 16, kRowsPerWarp = 32 / kTpr;
  if (p.max_new <= kRowsPerWarp) {
    const int pages_per = p.max_new == 1 ? 1 : 2;  // pages of 16 tokens at least
    const int64_t kv_warps = (int64_t)p.batch * pages_per * 2 * p.hkv;
    const int64_t q_rows = p.q != nullptr ? (int64_t)p.batch * p.max_new * p.hq : 0;
    const int64_t warps = kv_warps + (q_rows + kRowsPerWarp - 1) / kRowsPerWarp;
    const int64_t blocks = (warps + 3) / 4;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_ahead(append_steps_kernel<D, kF8, kAxes>, dim3((unsigned)blocks), 128, 0, stream, p,
                        pages_per, kv_warps);
  }
  const int need = kTpr << p.page_shift;  // threads that hold a page in one pass
  const int most = need <= 512 ? 256 : 512;
  const int threads = need < most ? need : most, passes = need / threads;
  const int q_shift = log2_of(threads / kTpr);
  const int64_t kv_blocks = ((p.total_new >> p.page_shift) + 2 * (int64_t)p.batch) * 2 * p.hkv;
  const int q_groups = (p.hq + kQHeads - 1) / kQHeads;
  const int64_t q_blocks =
      p.q != nullptr ? ((p.total_new >> q_shift) + 2 * (int64_t)p.batch) * q_groups : 0;
  if (kv_blocks + q_blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)(kv_blocks + q_blocks);
  // rounded up: grid * q_share / 2^32 is then q_blocks exactly, for grid < 2^32
  const uint64_t q_share = (((uint64_t)q_blocks << 32) + grid - 1) / grid;
  auto kernel = passes == 1   ? append_pages_kernel<D, kF8, 1, 256, kAxes>
                : most == 256 ? append_pages_kernel<D, kF8, 2, 256, kAxes>
                              : append_pages_kernel<D, kF8, 2, 512, kAxes>;
  return launch_ahead(kernel, dim3(grid), threads, 0, stream, p, q_share, q_shift, q_groups);
}

template <int D, bool kF8>
cudaError_t launch_positions(const KvAppendArgs& p, cudaStream_t stream) {
  return p.positions != nullptr ? launch_append<D, kF8, true>(p, stream)
                                : launch_append<D, kF8, false>(p, stream);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& args, cudaStream_t stream) {
  KvAppendArgs a = args;
  a.page_shift = log2_of(a.page_size);
  if (a.d == 64)
    return a.f8 ? launch_positions<64, true>(a, stream) : launch_positions<64, false>(a, stream);
  if (a.d == 128)
    return a.f8 ? launch_positions<128, true>(a, stream) : launch_positions<128, false>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace tts
