// Attention of a drafted tree of new tokens over the paged grouped-query cache.
//
// Request r's n new tokens are its last n cached rows. Token i sees the new tokens whose bits its
// mask has, and the cached ones before them (with a window: those of its position's window and the
// first ones); its position is past the cached tokens by the number of new tokens that it
// sees besides one (itself).
//
// A tree has more q rows per KV head than a decode step (16 to 64 tokens by the group's heads), so the
// products run on the tensor cores with the q rows as M = 128: S = Q K^T, O += P V, accumulators in
// TMEM, a softmax thread per q row. For KV head g the rows of its group (token-major) are blocks of
// 128, or 256 where requests have more; a unit is (request, g, row block), a tile kTK keys. All
// tiles of all units form one list, cut into equal runs, one per CTA (one CTA per SM); a
// unit cut by a run's border leaves unnormalised sums that a second launch joins in order. Roles:
//   warp 0       TMA producer: pages through the table into a ring of K tiles and one of V tiles
//   warp 1       tcgen05 issuer (TMEM: S0, S1 at columns 0 and 128, O0, O1 at 256 and 384)
//   warps 2, 3   V for the second product: e4m3 codes to fp16; rows that no token sees to zeros
//   warps 4..11  two softmax warpgroups. Up to 128 rows: both hold the same rows and take the tiles in
//                turn, each with its own running maximum, sum and accumulator, joined at the unit's
//                end. More rows: each holds 128 and takes every tile.
// Either way the products of one warpgroup run while the other's softmax does.
//
// e4m3 caches: K codes are multiplied as they are (kind::f8f6f4), with q as the sum of two e4m3
// values: a row is scaled by a power of two so that its largest value lies in [2^7, 2^8); hi has
// the leading 4 bits and lo the next 4, all of a bf16 value, down to 2^-9 of the row's largest; below
// that lo ends at 2^-10, 2^-17 of the largest. Widening K instead would read and write
// three times the tile's bytes in shared memory, whose rate is what the tensor core's operands
// leave least of. Weights are fp16 against V widened to fp16 (exactly): e4m3 weights, in two
// terms as well, would end at 2^-18 of the largest, and a flat tail of keys under a dominant one loses
// digits there. The value scale of a page rides in the exponent as in attn_decode.cu:
//   x_j = scale log2(e) sK q.k_j + log2 sV,   weights 2^(x_j - m), summed with 1 / sV.
// bf16 caches use bf16 products throughout. Sums and statistics are fp32.
//
// Code that a part runs once, or few tiles do, is kept short (loops that are not unrolled): three warps
// of different roles share an SM quarter's instruction cache, and what it does not hold is waited for.
// The q rows' conversion unrolled over four rows instead of one cost 16 large trees 10 us of 104.
//
// Measured (one GPU, CUDA graph; 16 requests x 20000 tokens, 4 KV heads of 128; reading the cache
// once at the rate of a copy takes 48 us in e4m3, 97 in bf16; products at the rate of a large bf16
// matrix product 0.34 us per row):
//   rows per KV head      32     128     256     512
//   e4m3, us            70.7    79.0     137     251
//   bf16, us             107     112     129     247
// Up to 128 rows over bf16 HBM bounds it (0.91 of the copy rate at 32 rows, 1.03 over 32 requests
// x 32768); over e4m3 the chain of a tile's S, weights, P V, of which each warpgroup has one under way.
// From 256 rows on that chain and the tensor core (0.65 of the rate above).
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tts {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kThreads = 384;
constexpr int kRows = 128;  // q rows of a tile (TMEM lanes)
// What the end of a unit costs (its sums, the next unit's first tile), in tiles of the list: 4 to 8 are
// within 5 % of one another on batches of 1 to 100 requests.
constexpr int kEndTiles = 7;
constexpr int kParts = 4;   // parts of a run that are described ahead
constexpr int kMinRun = 2;  // places of a run at least: a tile for each warpgroup
constexpr float kMinValueScale = 0x1p-80f;  // as in attn_decode.cu
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// kTwo: units of up to 256 rows, two q tiles.
template <bool F8, int D, bool kTwo>
struct Cfg {
  static constexpr int kRowBytes = D * (F8 ? 1 : 2);
  static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;  // one swizzled row
  static constexpr int kPanels = kRowBytes / kPanelBytes;
  static constexpr int kTK = 128;                    // keys per tile: whole pages
  static constexpr int kTileBytes = kTK * kRowBytes;       // K (or V) of one tile
  static constexpr int kQTiles = kTwo ? 2 : 1;
  // e4m3: the hi and the lo half one after the other, each kRows rows of one panel
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kWideBytes = F8 ? kTK * D * 2 : 0;  // V as fp16
  static constexpr int kWides = F8 ? 2 : 0;
  static constexpr int kLimit = 224 * 1024;  // of 227 KB: 1 KB to align, 2 of barriers and the rest
  static constexpr int kRing = (kLimit - kQTiles * kQBytes - kWides * kWideBytes) / (2 * kTileBytes);
  static constexpr int kStages = kRing < 8 ? kRing : 8;
  // A tile's scales are read until its weights are computed, two jobs behind its K's last reader.
  static constexpr int kMeta = kStages + 2;
  static constexpr int kSmemBytes =
      1024 + kQTiles * kQBytes + kWides * kWideBytes + kStages * 2 * kTileBytes;
  static constexpr int kPieces = F8 ? kTK / 16 : 1;
  static constexpr int kUnitRows = kQTiles * kRows;
  static_assert(kStages >= 2, "ring");
};

// Registers move from the warps that issue to the softmax warps, which hold a tile's scores: 128 x
// 104 + 256 x 200 = 64512 = 384 x 168, all that the block is launched with.
constexpr int kIssueRegs = 104, kSoftmaxRegs = 200;
constexpr int kLaunchRegs = (128 * kIssueRegs + 256 * kSoftmaxRegs + kThreads - 1) / kThreads;
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// kind::f16 with fp16 A and B, fp32 D; b_mn: B is N-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, uint32_t b_mn) {
  return (1u << 4) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// kind::f8f6f4 with e4m3 A and B, both K-major, fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss_f8_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate,
                                                uint32_t pred) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(pred)
      : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The two e4m3 codes in the low / high half of w as two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3_half(uint32_t w, int high) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)(high ? w >> 16 : w)));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
// Shared-memory address of 16-byte chunk c of row `row`, as TMA's swizzle and the matrix descriptors
// place it, in panels of `rows` rows (128-byte rows: chunk ^ row mod 8; 64-byte rows: chunk ^
// row / 2 mod 4).
template <int PB>
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int rows, int row, int c) {
  if constexpr (PB == 128)
    return base + (c >> 3) * (rows * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  else
    return base + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint32_t below(int n, int c0) {  // bits of columns c0 .. c0 + 31 under n
  const int b = n - c0;
  return b <= 0 ? 0u : b >= 32 ? kAll : (1u << b) - 1u;
}

// Which of the keys k0 .. k0 + 31 (word c of a tile) are seen: those before `base` from lo on (with a
// window) or among the first `sinks`, the new tokens in `mask`, on pages that are there.
__device__ __forceinline__ uint32_t seen_word(int k0, int c, int base, int window, int lo, int sinks,
                                              uint64_t mask, uint32_t pieces, int piece_shift) {
  uint32_t see = below(base, k0);
  if (window > 0) see &= ~below(lo, k0) | below(sinks, k0);
  const int sh = k0 - base;  // the word's first key among the new tokens
  if (sh > -32 && sh < 64) see |= (uint32_t)(sh >= 0 ? mask >> sh : mask << -sh);
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (!((pieces >> ((2 * c + u) >> piece_shift)) & 1u)) see &= ~(0xFFFFu << (16 * u));
  return see;
}

// Bounded wait of a converged warp in few instructions: every role has its own, and what the
// instruction cache does not hold is waited for as well. Sets *abort where it runs out.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort) {
  uint32_t since = 0;
  bool ok = true;
  if (!mbar_peek(bar, parity)) {
    while (!mbar_test(bar, parity)) {
      if (*abort) {
        ok = false;
        break;
      }
      uint32_t now;
      asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(now));
      if (since == 0) since = now | 1u;
      if ((int)(now - since) > (int)kWaitLimitNs) *abort = 1;
    }
  }
  return __all_sync(kAll, ok);
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
// Looks at three barriers at once.
__device__ __forceinline__ bool peek3(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, uint32_t c,
                                      uint32_t pc) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%5], %6;\n\t"
      "and.pred p, p, q;\n\tand.pred p, p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(a), "r"(pa), "r"(b), "r"(pb), "r"(c), "r"(pc)
      : "memory");
  return ok != 0;
}
// Two columns of a warp's TMEM lanes.
__device__ __forceinline__ void tmem_st2(uint32_t taddr, uint32_t a, uint32_t b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(a), "r"(b)
               : "memory");
}
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, uint32_t& a, uint32_t& b) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(taddr));
}

template <int kP>
struct Meta {  // of a tile, written by the producer
  float4 scale[kP];  // of a piece (a page, or the tile if pages are larger): its keys', log2 of its
                     // values', 1 / its values'
  int key0;          // first key
  uint32_t ok;       // bit i: piece i is there
  int clear;         // every row sees all of its keys
};
struct Part {  // tiles of one unit in a CTA's run, as the producer describes them
  int T;                 // tiles (0: the run is over)
  int q0, n, base;       // the request's first q row, its new tokens, its other keys
  int g, row0, rows;     // KV head, first row within the request, rows
  int whole_l, whole_r;  // the unit's first, its last tile are among them
  int c0;                // CTA that the unit began in, where it ends here
};

struct Params {
  const uint16_t* q;
  const int32_t* cu_q;  // null: one token per request
  const uint64_t* mask;
  const int32_t* page_tables;
  const int32_t* kv_lens;
  const float* k_scale;
  const float* v_scale;
  void* out;
  float* lse;
  // [2 * CTAs] parts: sums [D / 4][unit_rows] of four columns each (a row's thread writes beside its
  // neighbours'), then [unit_rows] {reference, denominator}
  float* parts;
  // [CTAs], of the unit that was begun in an earlier CTA and ended in this one: {first CTA
  // (-1: no such unit), rows, first row within the request, g}
  int4* jobs;
  int* job_q0;  // and the request's first q row
  uint32_t* dev_status;
  int total_q, max_keys;
  int batch, max_q, hq, hkv, group, num_pages, max_pages, page_size, page_shift, window, sinks;
  float scale_log2;
  int out_bf16, ctas, unit_rows;
};

// A request as the kernel sees it: its tokens, its visible keys as two runs of tiles (first
// tokens, window) and the number of units per head.
struct Req {
  int n, L, lo, sinks;  // new tokens, keys, first key of the widest window (0: none), first keys kept
  int st, lt, nt, rt;   // tiles of the first keys, first tile of the window, tiles, row blocks
  int q0;               // first q row
};
template <int TK>
__device__ __forceinline__ Req load_req(const Params& p, int b, uint32_t* bad) {
  Req r;
  int q1 = b + 1;
  r.q0 = b;
  if (p.cu_q != nullptr) {
    r.q0 = p.cu_q[b];
    q1 = p.cu_q[b + 1];
  }
  r.L = p.kv_lens[b];
  r.n = 0;
  if (r.q0 < 0 || q1 < r.q0 || q1 > p.total_q || q1 - r.q0 > p.max_q)
    *bad |= kDevBadArg;
  else
    r.n = q1 - r.q0;
  if (r.L < 0 || r.L > p.max_keys) {
    *bad |= kDevIndexRange;
    r.L = 0;  // its rows see no key
  }
  // keys and window are at most 2^30, so nothing here leaves 32 bits
  r.lo = p.window > 0 ? max(r.L - r.n + 1 - p.window, 0) : 0;
  r.sinks = min(p.sinks, r.lo);
  r.lt = (int)((unsigned)r.lo / TK);
  r.st = min((int)((unsigned)(r.sinks + TK - 1) / TK), r.lt);
  r.nt = max(r.st + (int)((unsigned)(r.L + TK - 1) / TK) - r.lt, 1);  // 1: an empty tile, zeros
  r.rt = (r.n * p.group + p.unit_rows - 1) / p.unit_rows;
  return r;
}
// Places of the list that a tile of a request's last row block takes: two where it has more than 128
// rows, which both warpgroups then go through (ragged trees of up to 155 rows, window 4096: 67 us
// with one place each, 53 with two).
__device__ __forceinline__ int last_weight(const Params& p, int n, int unit_rows) {
  const int rows = n * p.group;
  return (rows - 1) % unit_rows >= kRows ? 2 : 1;
}
// Places of the list that a request takes: its last row block may have up to 128 rows.
template <int kQTiles>
__device__ __forceinline__ int places_of(const Params& p, const Req& r) {
  if (r.rt == 0) return 0;
  return p.hkv * ((r.rt - 1) * r.nt * kQTiles + r.nt * last_weight(p, r.n, kQTiles * kRows) +
                  r.rt * kEndTiles);
}
// The list cut into runs of `len` or, the first `more` of them, one more place.
struct Runs {
  int runs, len, more;
  __device__ __forceinline__ Runs(int total, int ctas) {
    runs = min(max((int)((unsigned)total / kMinRun), 1), ctas);
    len = (int)((unsigned)total / (unsigned)runs);
    more = total - len * runs;
  }
  __device__ __forceinline__ int cta_of(int place) const {
    const int longer = more * (len + 1);  // places of the runs with one more
    return place < longer ? (int)((unsigned)place / (unsigned)(len + 1))
                          : more + (int)((unsigned)(place - longer) / (unsigned)len);
  }
};
__device__ __forceinline__ int warp_scan(int x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// A place in a ring of N slots and the parity of its current round.
template <int N>
struct Ring {
  int at = 0;
  uint32_t odd = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      odd ^= 1;
    }
  }
};
// Bits of new tokens that are there: m < n and a key of its own (a length under n has none for some).
__device__ __forceinline__ uint64_t present(int n, int base) {
  uint64_t m = n >= 64 ? ~0ull : (1ull << n) - 1;
  if (base < 0) m = -base >= 64 ? 0 : m >> -base << -base;
  return m;
}

template <bool F8, int D, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const Params p) {
  using C = Cfg<F8, D, kTwo>;
  constexpr int TK = C::kTK, S = C::kStages, PB = C::kPanelBytes;
  extern __shared__ uint8_t smem_raw[];
  // Of a part: described, its description read. Of a tile: K and V landed; their slots free (K's
  // products done; V's products done, or its codes widened: K's place is filled again a product earlier);
  // V ready for its product (widened, or cleared); its scales written. Of a warpgroup: scores, weights
  // of a tile's first 64 keys, all weights, sums. Of a part: the q tile written that a warpgroup's
  // scores read; every score read (the q tiles may be overwritten, and the columns that statistics
  // go through); the second warpgroup's statistics.
  __shared__ __align__(8) uint64_t bar_part[kParts], bar_part_empty[kParts], bar_k[S], bar_v[S],
      bar_k_empty[S], bar_v_empty[S], bar_ready[S], bar_meta[C::kMeta], bar_s[2], bar_half[2],
      bar_p[2], bar_o[2], bar_q[2], bar_q_empty, bar_ml, bar_drain;
  __shared__ __align__(16) Meta<C::kPieces> s_meta[C::kMeta];
  __shared__ Part s_part[kParts];
  __shared__ uint8_t s_ex[C::kUnitRows];  // e4m3: the exponent that a q row was scaled by
  __shared__ int s_scan[kThreads / 32], s_b, s_off, s_abort;
  __shared__ uint32_t s_tmem;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sq = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t wide = sq + C::kQTiles * C::kQBytes;
  const uint32_t ring = wide + C::kWides * C::kWideBytes;
  auto sK = [&](int st) -> uint32_t { return ring + st * 2 * C::kTileBytes; };
  auto sV = [&](int st) -> uint32_t { return ring + st * 2 * C::kTileBytes + C::kTileBytes; };
  volatile int* abort_flag = &s_abort;

  if (tid == 0) {
    prefetch_tmap(&map_k);  // on their way while the lengths are read
    prefetch_tmap(&map_v);
    s_abort = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&bar_k[i]), 1);
      mbar_init(smem_u32(&bar_v[i]), 1);
      mbar_init(smem_u32(&bar_k_empty[i]), 1);
      mbar_init(smem_u32(&bar_v_empty[i]), F8 ? 2 : 1);  // both warps that widen it
      mbar_init(smem_u32(&bar_ready[i]), 2);
    }
    for (int i = 0; i < C::kMeta; ++i) mbar_init(smem_u32(&bar_meta[i]), 1);
    for (int i = 0; i < kParts; ++i) {
      mbar_init(smem_u32(&bar_part[i]), 1);
      mbar_init(smem_u32(&bar_part_empty[i]), kThreads / 32 - 1);  // every warp but the producer
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_s[i]), 1);
      mbar_init(smem_u32(&bar_half[i]), kRows);
      mbar_init(smem_u32(&bar_p[i]), kRows);
      mbar_init(smem_u32(&bar_o[i]), 1);
      mbar_init(smem_u32(&bar_q[i]), 2 * kRows);
    }
    mbar_init(smem_u32(&bar_q_empty), 8);
    mbar_init(smem_u32(&bar_ml), kRows);
    mbar_init(smem_u32(&bar_drain), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  wait_for_prior_grids();
  if (tid == 0) p.jobs[blockIdx.x] = make_int4(-1, 0, 0, 0);

  // ---- this CTA's run [t0, t1) of the list of tiles, and the request it begins in
  uint32_t bad = 0;
  int total = 0, t0 = 0, t1 = 0;
  auto split = [&]() -> bool {
    if (total == 0) return false;
    const Runs cut(total, p.ctas);
    if ((int)blockIdx.x >= cut.runs) return false;
    t0 = blockIdx.x * cut.len + min((int)blockIdx.x, cut.more);
    t1 = t0 + cut.len + ((int)blockIdx.x < cut.more ? 1 : 0);
    return true;
  };
  auto block_scan = [&](int v, int* sum) -> int {  // inclusive
    const int x = warp_scan(v, lane);
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
  int b = 0, off = 0;
  bool work;
  if (p.batch <= 32) {  // every warp for itself
    const int v = lane < p.batch ? places_of<C::kQTiles>(p, load_req<TK>(p, lane, &bad)) : 0;
    const int incl = warp_scan(v, lane);
    total = __shfl_sync(kAll, incl, 31);
    work = split();
    if (work) {
      b = __ffs(__ballot_sync(kAll, incl > t0)) - 1;
      off = t0 - __shfl_sync(kAll, incl - v, b);
    }
    if (warp != 0) bad = 0;
  } else {
    for (int base = 0; base < p.batch; base += kThreads) {
      const int i = base + tid;
      int sum;
      block_scan(i < p.batch ? places_of<C::kQTiles>(p, load_req<TK>(p, i, &bad)) : 0, &sum);
      total += sum;
    }
    work = split();
    uint32_t again = 0;
    for (int base = 0, carry = 0; work && base < p.batch && carry <= t0; base += kThreads) {
      const int i = base + tid;
      const int v = i < p.batch ? places_of<C::kQTiles>(p, load_req<TK>(p, i, &again)) : 0;
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
  }
  if (blockIdx.x == 0 && bad && p.dev_status != nullptr) atomicOr(p.dev_status, bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  if (!work) {  // the same for the block
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  const int piece = p.page_size, n_pieces = TK / piece;  // keys per TMA box, a page; pages of a tile
  const int piece_shift = 31 - __clz(piece >> 4);  // 16 keys -> piece
  // The next part of the run, as the producer describes it to the other warps (false: there is none),
  // where it stays until the warp is done with it: registers are scarce.
  Ring<kParts> pslot;
  auto next_part = [&]() -> bool {
    return wait_for(smem_u32(&bar_part[pslot.at]), pslot.odd, abort_flag) && s_part[pslot.at].T > 0;
  };
  auto part_done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar_part_empty[pslot.at]));
    pslot.next();
  };

  if (warp < 4) {
    give_registers<kIssueRegs>();
    if (warp == 0) {
      // ------------------------------------------------------------------ producer
      // Walks the run. What it does for a tile must take well under the 1400 (heads of 64: 700) cycles
      // that HBM takes for an SM's share of it.
      Req r = load_req<TK>(p, b, &bad);
      int left = t1 - t0, parts = 0;
      int g, rt, at0;  // place within the unit
      {  // the run's first unit, perhaps from its middle
        const int full = r.nt * C::kQTiles + kEndTiles;  // places of a full row block
        const int head = (int)((unsigned)places_of<C::kQTiles>(p, r) / (unsigned)p.hkv);
        g = (int)((unsigned)off / (unsigned)head);
        at0 = off - g * head;
        rt = min((int)((unsigned)at0 / (unsigned)full), r.rt - 1);
        at0 -= rt * full;
      }
      int it = 0;
      Ring<S> slot;
      Ring<C::kMeta> mslot;
      // Of page cache_at + lane of request cache_b: the page, for head cache_g its key scale, log2 and
      // inverse of its value scale, and whether they are in range. The next 32 pages' are on their way.
      int cache_b = -1, cache_at = 0, cache_g = -1, page = -1, page_next = -1;
      bool fine = true;
      float ks = 1.f, vl = 0.f, vi = 1.f, sk_next = 1.f, sv_next = 1.f;
      bool asked = false;  // for the next pages' scales
      auto page_of = [&](int first) -> int {
        const int lp = first + lane;
        const int pg = lp < p.max_pages ? p.page_tables[(int64_t)b * p.max_pages + lp] : -1;
        return pg < p.num_pages ? pg : -1;  // < 0: none
      };
      auto scales_of = [&](int pg, float& sk, float& sv) {
        sk = sv = 1.f;
        if (pg >= 0) {
          sk = p.k_scale[(int64_t)pg * p.hkv + g];
          sv = p.v_scale[(int64_t)pg * p.hkv + g];
        }
      };
      bool ok = true;
      auto describe = [&](const Part& q) -> bool {
        if (parts >= kParts && !wait_for(smem_u32(&bar_part_empty[pslot.at]), pslot.odd ^ 1, abort_flag))
          return false;
        if (lane == 0) {
          s_part[pslot.at] = q;
          mbar_arrive(smem_u32(&bar_part[pslot.at]));
        }
        __syncwarp();
        pslot.next();
        ++parts;
        return true;
      };
      while (ok && left > 0) {
        // A unit whose warpgroups each take every tile counts a tile as two places: tile x begins at
        // place x weight. Runs have two places at least, so that none lies between two tiles.
        const int weight = rt == r.rt - 1 ? last_weight(p, r.n, C::kUnitRows) : C::kQTiles;
        const int begin = t1 - left - at0;  // list place of the unit's first tile
        const int x0 = (at0 + weight - 1) >> (weight - 1);
        const int x1 = min(r.nt, (at0 + left + weight - 1) >> (weight - 1));
        left -= min(r.nt * weight + kEndTiles - at0, left);
        at0 = 0;
        const int base = r.L - r.n;
        if (x0 < x1) {  // else the run begins behind the unit's last tile
          Part q;
          q.T = x1 - x0;
          q.q0 = r.q0;
          q.n = r.n;
          q.base = base;
          q.g = g;
          q.row0 = rt * C::kUnitRows;
          q.rows = min(r.n * p.group - q.row0, C::kUnitRows);
          q.whole_l = x0 == 0;
          q.whole_r = x1 == r.nt;
          q.c0 = 0;
          if (!q.whole_l && q.whole_r) q.c0 = Runs(total, p.ctas).cta_of(begin);  // the unit ends here
          ok = describe(q);
        }
        // every row sees the keys of a tile in front of `base` and, with a window, from clear_lo on (or
        // among the first ones)
        const int clear_lo = p.window > 0 ? base + r.n - p.window : 0;
        for (int x = x0; ok && x < x1; ++x, ++it, slot.next(), mslot.next()) {
          const int key0 = (x < r.st ? x : r.lt + x - r.st) * TK, st = slot.at;
          const int pg0 = key0 >> p.page_shift;
          if (cache_b != b || cache_g != g || pg0 < cache_at || pg0 + n_pieces > cache_at + 32) {
            float sk = 1.f, sv = 1.f;
            if (cache_b == b && cache_g == g && pg0 == cache_at + 32) {
              page = page_next;
              if (F8 && !asked) scales_of(page, sk_next, sv_next);
              sk = sk_next;
              sv = sv_next;
            } else {
              page = page_of(pg0);
              if (F8) scales_of(page, sk, sv);
            }
            cache_b = b;
            cache_at = pg0;
            cache_g = g;
            page_next = page_of(pg0 + 32);
            asked = false;
            if constexpr (F8) {
              fine = sk > 0.f && sk < INFINITY && sv >= kMinValueScale && sv < INFINITY;
              ks = sk;
              vl = fine ? log2f(sv) : 0.f;
              vi = fine ? 1.f / sv : 0.f;
            }
          } else if (F8 && !asked) {
            scales_of(page_next, sk_next, sv_next);
            asked = true;
          }
          // Lane cache's page that is piece k of the tile: keys [a, a + piece)
          const int k = lane - (pg0 - cache_at), a = key0 + k * piece;
          const bool seen = k >= 0 && k < n_pieces && a < r.L && (a + piece > r.lo || a < r.sinks);
          const bool there = seen && page >= 0;
          const uint32_t sent = __ballot_sync(kAll, there);
          const uint32_t use = (F8 ? __ballot_sync(kAll, there && fine) : sent) >> (pg0 - cache_at);
          const uint32_t full_k = smem_u32(&bar_k[st]), full_v = smem_u32(&bar_v[st]);
          const uint32_t bytes = __popc(sent) * piece * C::kRowBytes;
          const int slab = page * p.hkv + g;
          auto load = [&](uint32_t to, const CUtensorMap* map, uint32_t bar) {
            if (there) {
#pragma unroll
              for (int pn = 0; pn < C::kPanels; ++pn)
                tma_load_3d(to + pn * TK * PB + k * piece * PB, map, bar, pn * 64, 0, slab);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          };
          if (it >= S) {
            ok = wait_for(smem_u32(&bar_k_empty[st]), slot.odd ^ 1, abort_flag);
            if (!ok) break;
          }
          load(sK(st), &map_k, full_k);
          Meta<C::kPieces>& meta = s_meta[mslot.at];
          if constexpr (F8) {
            if (k >= 0 && k < n_pieces)  // pieces that are not used stay neutral
              meta.scale[k] = there && fine ? make_float4(ks, vl, vi, 0.f) : make_float4(1.f, 0.f, 0.f, 0.f);
          }
          if (seen && !(there && fine) && p.dev_status != nullptr)  // or no scale of a written page
            atomicOr(p.dev_status, there ? kDevBadArg : kDevIndexRange);
          if (lane == 0) {
            meta.key0 = key0;
            meta.ok = use;
            meta.clear = use == (1u << n_pieces) - 1u && key0 + TK <= base &&
                         (p.window == 0 || key0 >= clear_lo || key0 + TK <= p.sinks);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_meta[mslot.at]));
          if (it >= S) {
            ok = wait_for(smem_u32(&bar_v_empty[st]), slot.odd ^ 1, abort_flag);
            if (!ok) {
              if (lane == 0) mbar_arrive(full_v);  // nothing is on its way
              ++it;
              break;
            }
          }
          load(sV(st), &map_v, full_v);
        }
        if (left > 0 && ++rt == r.rt) {
          rt = 0;
          if (++g == p.hkv) {
            g = 0;
            do r = load_req<TK>(p, ++b, &bad);  // requests without new tokens have no units
            while (r.rt == 0);
          }
        }
      }
      Part none;
      none.T = 0;
      if (ok) describe(none);
      // Copies in flight must land before the CTA can exit, also when a wait ran out.
      for (int i = it > S ? it - S : 0; i < it; ++i) {
        mbar_wait(smem_u32(&bar_k[i % S]), (i / S) & 1, nullptr, nullptr);
        mbar_wait(smem_u32(&bar_v[i % S]), (i / S) & 1, nullptr, nullptr);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------ tcgen05 issuer
      const uint32_t e = elect_one();
      auto s_t = [&](int w) -> uint32_t { return tmem + w * 128; };
      auto o_t = [&](int w) -> uint32_t { return tmem + 256 + w * 128; };
      constexpr uint32_t kKSbo = PB * 8;  // eight rows
      constexpr SmemLayout kLay = PB == 128 ? kSw128 : kSw64;
      auto issue_s = [&](int w, int tile, int st) {
        const uint64_t qd = smem_desc(sq + tile * C::kQBytes, 16, kKSbo, kLay);
        const uint64_t kd = smem_desc(sK(st), 16, kKSbo, kLay);
        if constexpr (F8) {
          constexpr uint32_t idesc = idesc_e4m3_f32(kRows, TK);
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              mma_ss_f8_elect(s_t(w), qd + ((half * kRows * PB + k * 32) >> 4), kd + ((k * 32) >> 4),
                              idesc, half + k > 0, e);
        } else {
          constexpr uint32_t idesc = idesc_bf16_f32(kRows, TK, 0, 0);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss_elect(s_t(w), qd + (((k / 4) * kRows * 128 + (k % 4) * 32) >> 4),
                         kd + (((k / 4) * TK * 128 + (k % 4) * 32) >> 4), idesc, k > 0, e);
        }
      };
      auto issue_o = [&](int w, uint32_t v, bool acc, auto half) {
        constexpr int k0 = decltype(half)::value * (TK / 32);
        const uint64_t vd = smem_desc(v, TK * 128, 1024, kSw128);
        constexpr uint32_t idesc = F8 ? idesc_f16_f32(kRows, D, 1) : idesc_bf16_f32(kRows, D, 0, 1);
#pragma unroll
        for (int k = k0; k < k0 + TK / 32; ++k)
          mma_ts_elect(o_t(w), s_t(w) + k * 8, vd + ((k * 16 * 128) >> 4), idesc, acc || k > 0, e);
      };
      Ring<S> kslot, vslot;   // of the next tile whose S, whose P V is issued
      uint32_t wide_at = 0;   // e4m3: its widened V
      uint32_t odd_p[2] = {0, 0}, odd_q = 0;  // parities of the phases waited for next
      bool ok = true;
      while (ok && next_part()) {
        const bool alt = !kTwo || s_part[pslot.at].rows <= kRows;
        const int J = alt ? s_part[pslot.at].T : 2 * s_part[pslot.at].T;
        part_done();
        // Job i: warpgroup i % 2, and tile i, or i / 2 where each warpgroup takes every tile. The product
        // of job i - 2's weights comes in front of job i's scores, which overwrite them. A part's first
        // scores run while the sums of the part before are read: its first product, which overwrites
        // them, waits for weights that the warpgroup computes after it read them (the second warpgroup's
        // sums, read by the first where they take turns, as well: its job comes after job 0).
        auto step = [&](auto which, int i) -> bool {
          constexpr int w = decltype(which)::value;
          const bool pv = i >= 2 && i < J + 2, qk = i < J;
          if (!pv && !qk) return true;
          // Everything the step needs is looked at together: a look takes as long as an issue.
          const uint32_t bar_a = pv ? smem_u32(&bar_half[w]) : smem_u32(&bar_q[w]);
          const uint32_t bar_b = pv ? smem_u32(&bar_ready[vslot.at]) : bar_a;
          const uint32_t bar_c = qk ? smem_u32(&bar_k[kslot.at]) : bar_a;
          const uint32_t odd_a = pv ? odd_p[w] : odd_q, odd_b = pv ? vslot.odd : odd_a,
                         odd_c = qk ? kslot.odd : odd_a;
          uint32_t since = 0;
          while (!__all_sync(kAll, peek3(bar_a, odd_a, bar_b, odd_b, bar_c, odd_c))) {
            if (__any_sync(kAll, *abort_flag)) return false;
            uint32_t now;
            asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(now));
            if (since == 0) since = now | 1u;
            if ((int)(now - since) > (int)kWaitLimitNs) *abort_flag = 1;
          }
          tc_fence_after();
          if (pv) {
            // the products with the first 64 weights run while the others are computed
            const uint32_t v = F8 ? wide + wide_at * C::kWideBytes : sV(vslot.at);
            issue_o(w, v, i >= 4, std::integral_constant<int, 0>());
            if (!wait_for(smem_u32(&bar_p[w]), odd_p[w], abort_flag)) return false;
            tc_fence_after();
            issue_o(w, v, true, std::integral_constant<int, 1>());
            odd_p[w] ^= 1;
            if (alt || w == 1) {
              if (!F8) mma_commit_elect(smem_u32(&bar_v_empty[vslot.at]), e);
              vslot.next();
              wide_at ^= 1;
            }
          }
          if (qk) {
            issue_s(w, alt ? 0 : w, kslot.at);
            // who sees it hands K back, and widens the next V
            mma_commit_elect(smem_u32(&bar_s[w]), e);
            if (alt || w == 1) kslot.next();
          }
          if (pv && i >= J) mma_commit_elect(smem_u32(&bar_o[w]), e);
          return true;
        };
        for (int i = 0; ok && i < J + 2; i += 2)
          ok = step(std::integral_constant<int, 0>(), i) && step(std::integral_constant<int, 1>(), i + 1);
        odd_q ^= 1;
      }
      // Every product is complete before TMEM is freed.
      mma_commit_elect(smem_u32(&bar_drain), e);
      mbar_wait(smem_u32(&bar_drain), 0, nullptr, p.dev_status);
    } else {
      // ------------------------------------------------------------------ V for the second product
      Ring<S> slot;
      Ring<C::kMeta> mslot;
      uint32_t wide_at = 0, odd_s[2] = {0, 0};  // e4m3: the widened V, parities of the next scores
      bool ok = true;
      while (ok && next_part()) {
        const Part q = s_part[pslot.at];
        part_done();
        const bool alt = !kTwo || q.rows <= kRows;
        // new tokens that some token sees, and the first key of the windows
        const uint64_t here = present(q.n, q.base);
        uint64_t any = 0;
        int least = 64;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (lane + 32 * k < q.n) {
            const uint64_t m = p.mask[q.q0 + lane + 32 * k];
            any |= m;
            least = min(least, max(__popcll(m & (q.n >= 64 ? ~0ull : (1ull << q.n) - 1)) - 1, 0));
          }
        any = here & ((uint64_t)__reduce_or_sync(kAll, (uint32_t)any) |
                      (uint64_t)__reduce_or_sync(kAll, (uint32_t)(any >> 32)) << 32);
        least = __reduce_min_sync(kAll, least);
        const int lo = p.window > 0 ? max(q.base + least + 1 - p.window, 0) : 0;
        const int kept = min(p.sinks, lo);
        for (int x = 0; x < q.T; ++x, slot.next(), mslot.next(), wide_at ^= 1) {
          const int st = slot.at;
          ok = wait_for(smem_u32(&bar_v[st]), slot.odd, abort_flag);  // and the tile's description written
          // e4m3: with the tile's own scores (the first of them) the products with the V two tiles before
          // are complete, whose place this one takes; the next scores of that warpgroup wait for it.
          if constexpr (F8) {
            const bool second = alt && (x & 1);
            ok = ok && wait_for(smem_u32(&bar_s[second]), second ? odd_s[1] : odd_s[0], abort_flag);
            if (second || !alt) odd_s[1] ^= 1;
            if (!second) odd_s[0] ^= 1;
          }
          if (!ok) break;
          const uint32_t okp = s_meta[mslot.at].ok;
          const int key0 = s_meta[mslot.at].key0;
          const bool all = s_meta[mslot.at].clear;
          // words of the rows that some token sees, one a lane: the others' V is cleared
          const int word = lane & 3;
          const uint32_t mine = all ? kAll
                                    : seen_word(key0 + 32 * word, word, q.base, p.window, lo, kept, any,
                                                okp, piece_shift);
          auto clear_unseen = [&](auto clear, int row0, int step) {
            if (all) return;
#pragma unroll 1
            for (int c = 0; c < TK / 32; ++c) {
              const uint32_t see = __shfl_sync(kAll, mine, c);
              if (see == kAll) continue;
#pragma unroll 1
              for (int row = row0; row < 32; row += step)
                if (!((see >> row) & 1u)) clear(32 * c + row);
            }
          };
          if constexpr (F8) {
            const uint32_t from = sV(st), to = wide + wide_at * C::kWideBytes;
            // A thread's chunks of 16 codes lie kStep rows apart in one column: the swizzle is the
            // same for all of them. kDeep are on their way at a time.
            constexpr int kCpr = D / 16, kStep = 64 / kCpr, kDeep = 4;
            static_assert(TK % (kStep * kDeep) == 0 && kStep % 8 == 0, "chunks");
            const int i0 = (warp - 2) * 32 + lane, row0 = i0 / kCpr, c = i0 % kCpr;
            // the second panel's lanes store the other chunk first: eight lanes, all banks
            const int odd = c >> 2 & 1;
            const uint32_t src = chunk_at<PB>(from, TK, row0, c);
            const uint32_t dst0 = chunk_at<128>(to, TK, row0, 2 * c + odd),
                           dst1 = chunk_at<128>(to, TK, row0, 2 * c + 1 - odd);
#pragma unroll 1
            for (int k0 = 0; k0 < TK / kStep; k0 += kDeep) {
              uint4 v[kDeep];
#pragma unroll
              for (int k = 0; k < kDeep; ++k) v[k] = lds128(src + (k0 + k) * kStep * PB);
#pragma unroll
              for (int k = 0; k < kDeep; ++k) {
                const uint32_t x4[4] = {odd ? v[k].z : v[k].x, odd ? v[k].w : v[k].y,
                                        odd ? v[k].x : v[k].z, odd ? v[k].y : v[k].w};
                sts128(dst0 + (k0 + k) * kStep * 128,
                       make_uint4(e4m3_half(x4[0], 0), e4m3_half(x4[0], 1), e4m3_half(x4[1], 0),
                                  e4m3_half(x4[1], 1)));
                sts128(dst1 + (k0 + k) * kStep * 128,
                       make_uint4(e4m3_half(x4[2], 0), e4m3_half(x4[2], 1), e4m3_half(x4[3], 0),
                                  e4m3_half(x4[3], 1)));
              }
            }
            clear_unseen(
                [&](int row) {  // whole steps from row0
                  sts128(dst0 + (row - row0) * 128, make_uint4(0, 0, 0, 0));
                  sts128(dst1 + (row - row0) * 128, make_uint4(0, 0, 0, 0));
                },
                row0, kStep);
            fence_proxy_async_smem();
          } else if (!all) {
            const int i0 = (warp - 2) * 32 + lane, c = i0 % (D / 8);
            clear_unseen([&](int row) { sts128(chunk_at<PB>(sV(st), TK, row, c), make_uint4(0, 0, 0, 0)); },
                         i0 / (D / 8), 64 / (D / 8));
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&bar_ready[st]));
            if (F8) mbar_arrive(smem_u32(&bar_v_empty[st]));
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    take_registers<kSoftmaxRegs>();
    constexpr float kThr = F8 ? 4.f : 8.f;    // the reference moves when exceeded by 2^kThr
    // Weights are held times 2^kBias: at most 2^15 in fp16, where three roundings of scores below 2^23 (in
    // units of log2; steps of 1/2) add up to 3/4.
    constexpr float kBias = F8 ? 11.f : 0.f;
    const int w = (warp - 4) >> 2;
    const int lane_row = ((warp & 3) << 5) + lane;  // TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t S_row = tmem + w * 128 + lane_off;
    Ring<S> kslot;         // of the part's next tile
    Ring<C::kMeta> mslot;
    // parities of the phases waited for next: own scores, own sums, the other's sums, its statistics,
    // q tiles, the scores of the part before
    uint32_t odd_s = 0, odd_o = 0, odd_other = 0, odd_ml = 0, odd_q = 0, odd_empty = 1;
    // A q tile is written by one warpgroup: its own, or, where they take turns, by the second while the
    // first writes the sums of the part before (a run's first q tile by both). D / 16 lanes to a row, 16
    // values each, which lie in shared memory as copied (e4m3: in the place of the row's two halves) until
    // the lane turns them into its 16 codes of either half.
    constexpr int kLanes = D / 16, kPass = 4 * 32 / kLanes;
    bool first = true;  // part
    uint64_t seen = 0;  // this thread's row's mask
    auto takes_turns = [&](const Part& q) -> bool { return !kTwo || q.rows <= kRows; };
    const int q_lane = lane % kLanes, q_row = (warp & 3) * (32 / kLanes) + lane / kLanes;
    auto raw_at = [&](uint32_t to, int row, int i) -> uint32_t {  // i-th of the lane's two pieces
      if constexpr (F8)
        return chunk_at<PB>(to + (2 * q_lane >= kLanes ? kRows * PB : 0), kRows, row,
                            (2 * q_lane + i) % kLanes);
      else
        return chunk_at<PB>(to, kRows, row, 2 * q_lane + i);
    };
    auto ask = [&](const Part& q) -> bool {  // of the next part
      const bool alt = takes_turns(q);
      const int r0 = alt ? 0 : w * kRows;
      if (r0 + lane_row < q.rows) seen = p.mask[q.q0 + (q.row0 + r0 + lane_row) / p.group];
      if (alt && w == 0 && !first) return true;
      if (!first && !wait_for(smem_u32(&bar_q_empty), odd_empty, abort_flag)) return false;
      const uint32_t to = sq + (r0 ? C::kQBytes : 0);
      const int share = alt && first;
#pragma unroll 1
      for (int row = q_row + share * w * kPass; row - lane / kLanes < q.rows - r0 && row < kRows;
           row += kPass << share) {
        const bool in = r0 + row < q.rows;
        const int rr = q.row0 + r0 + row, tok = in ? rr / p.group : 0;
        const int64_t at = (int64_t)(q.q0 + tok) * p.hq + q.g * p.group + (rr - tok * p.group);
        const uint16_t* src = in ? p.q + at * D + q_lane * 16 : p.q;
        cp_async_16(raw_at(to, row, 0), src, in ? 16 : 0);
        cp_async_16(raw_at(to, row, 1), src + 8, in ? 16 : 0);
      }
      return true;
    };
    bool ok = next_part() && ask(s_part[pslot.at]);
    while (ok) {
      const Part& q = s_part[pslot.at];
      const bool alt = takes_turns(q);
      const int share = alt && first;
      if (!alt || w == 1 || share) {
        cp_async_wait_all();
        if constexpr (F8) {
          const int r0 = alt ? 0 : w * kRows;
          const uint32_t to = sq + (r0 ? C::kQBytes : 0);
#pragma unroll 1
          for (int row = q_row + share * w * kPass; row - lane / kLanes < q.rows - r0 && row < kRows;
               row += kPass << share) {
            const uint4 v0 = lds128(raw_at(to, row, 0)), v1 = lds128(raw_at(to, row, 1));
            const uint32_t u[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            uint32_t top = 0;  // largest |q| of the row, as bf16 bits
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t m = u[i] & 0x7FFF7FFFu;
              top = max(top, max(m & 0xFFFFu, m >> 16));
            }
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(kAll, top, d));
            const int ex = max((int)(top >> 7), 27);  // biased exponent; q' = q 2^(7 - e) < 2^8
            const float up = __uint_as_float((uint32_t)(261 - ex < 1 ? 1 : 261 - ex) << 23);
            if (q_lane == 0) s_ex[r0 + row] = (uint8_t)ex;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a = __uint_as_float(u[i] << 16) * up,
                          b2 = __uint_as_float(u[i] & 0xFFFF0000u) * up;
              const uint32_t h = cvt_e4m3x2(a, b2);
              const float2 back = e4m3x2_to_float2((uint16_t)h);
              const uint32_t low = cvt_e4m3x2(a - back.x, b2 - back.y);
              hi[i / 2] = i & 1 ? hi[i / 2] | h << 16 : h;
              lo[i / 2] = i & 1 ? lo[i / 2] | low << 16 : low;
            }
            __syncwarp();  // the row is read
            const uint32_t dst = chunk_at<PB>(to, kRows, row, q_lane);
            sts128(dst, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            sts128(dst + kRows * PB, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          }
        }
        fence_proxy_async_smem();
        const uint32_t n = 2 - share;
        mbar_arrive_n(smem_u32(&bar_q[w]), n);
        if (alt) mbar_arrive_n(smem_u32(&bar_q[w ^ 1]), n);
      }
      first = false;
      odd_empty ^= 1;
      // ---- this thread's q row: position, mask, factor of its scores
      const int row = lane_row + (alt ? 0 : w * kRows);
      const bool in = row < q.rows, live = row - lane < q.rows;
      uint64_t mask = in ? seen & (q.n >= 64 ? ~0ull : (1ull << q.n) - 1) : 0;
      const int pos = q.base + max(__popcll(mask) - 1, 0);
      mask &= present(q.n, q.base);
      float fac = p.scale_log2;
      if constexpr (F8) {
        ok = wait_for(smem_u32(&bar_q[w]), odd_q, abort_flag);  // the rows' exponents
        if (!ok) break;
        const int ex = in ? s_ex[row] : 127;
        fac *= __uint_as_float((uint32_t)(ex < 8 ? 1 : ex - 7) << 23);
      }
      odd_q ^= 1;
      // A tile's scores by a page's key scale. Kept above 0 where the product underflows (a row of zeros,
      // whose factor is 2^-107 of the scale, over a page of zeros, whose scale is 2^-60): hidden keys hold
      // -inf in front of it, and -inf times 0 is NaN. Products are below 2^25, so that a visible score stays
      // under 2^-101, which moves no weight. 0.3 to 1 % (16 x 20000 tokens, 32 rows 69.6 -> 70.4 us).
      auto factor = [&](float key_scale) -> float { return fmaxf(fac * key_scale, 0x1p-126f); };
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < q.T; ++j, mslot.next(), kslot.next()) {  // tile of the part
        if (alt && (j & 1) != w) continue;
        ok = wait_for(smem_u32(&bar_meta[mslot.at]), mslot.odd, abort_flag) &&
             wait_for(smem_u32(&bar_s[w]), odd_s, abort_flag);
        if (!ok) break;
        odd_s ^= 1;
        if (lane_row == 0 && (alt || w == 1)) mbar_arrive(smem_u32(&bar_k_empty[kslot.at]));
        __syncwarp();  // TMEM is read by converged warps
        if (!live) {  // no row of this warp is one of the unit's: what its lanes hold is never read
          mbar_arrive(smem_u32(&bar_half[w]));
          mbar_arrive(smem_u32(&bar_p[w]));
          continue;
        }
        tc_fence_after();
        const Meta<C::kPieces>& meta = s_meta[mslot.at];
        // Scores in the exp2 domain are s a + vl, with a and vl of the key's page; a > 0, so a page's
        // largest score has its largest s. They are read twice, for their maximum and for their weights.
        float tile_max = -INFINITY;
        if (meta.clear && (!F8 || piece_shift > 0)) {
          uint32_t x[32];
          float most[TK / 32];
#pragma unroll
          for (int c = 0; c < TK / 32; ++c) most[c] = tmem_ld32_max(S_row + c * 32, x);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < TK / 32; ++c) {
            if constexpr (F8) {
              const float4 sc = meta.scale[(2 * c) >> piece_shift];
              most[c] = fmaf(most[c], factor(sc.x), sc.y);
            }
            tile_max = fmaxf(tile_max, most[c]);
          }
        } else {
          // What a row does not see becomes -inf, in TMEM: a short loop, since such tiles are few and
          // code that is seldom run is waited for.
          const uint32_t okp = meta.ok;
#pragma unroll 1
          for (int c = 0; c < TK / 32; ++c) {
            const uint32_t see = seen_word(meta.key0 + 32 * c, c, q.base, p.window, pos + 1 - p.window,
                                           p.sinks, mask, okp, piece_shift);
            uint32_t x[32];
            tmem_ld32(S_row + c * 32, x);
            tmem_ld_wait();
            if (!__all_sync(kAll, see == kAll)) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((see >> i) & 1u)) x[i] = 0xFF800000u;
              tmem_st32(S_row + c * 32, x);
            }
            const float* s = reinterpret_cast<const float*>(x);
            if constexpr (F8) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float4 sc = meta.scale[(2 * c + u) >> piece_shift];
                tile_max = fmaxf(tile_max, fmaf(row_max<16>(s + 16 * u), factor(sc.x), sc.y));
              }
            } else {
              tile_max = fmaxf(tile_max, row_max<32>(s));
            }
          }
          tmem_st_wait();
        }
        if (!F8) tile_max *= fac;
        const bool resc = tile_max > m_ref + kThr;  // false for -inf
        float alpha = 1.f;
        if (resc) {
          alpha = ex2_approx(m_ref - tile_max);  // 0 from -inf
          l *= alpha;
          m_ref = tile_max;
        }
        __syncwarp();
        const float shift = m_ref == -INFINITY ? 0.f : kBias - m_ref;
        // ---- weights, packed in front of the scores that are still to be read
#pragma unroll 4
        for (int c = 0; c < TK / 32; ++c) {
          uint32_t x[32];
          tmem_ld32(S_row + c * 32, x);
          tmem_ld_wait();
          const float* s = reinterpret_cast<const float*>(x);
          uint32_t pk[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float a = fac, add = shift, inv = 1.f;
            if constexpr (F8) {
              const float4 sc = meta.scale[(2 * c + h) >> piece_shift];
              a = factor(sc.x);
              add = shift + sc.y;
              inv = sc.z;
            }
            const float2 a2 = make_float2(a, a), b2 = make_float2(add, add);
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              float2 y = ffma2(make_float2(s[16 * h + 2 * u], s[16 * h + 2 * u + 1]), a2, b2);
              y.x = ex2_approx(y.x);
              y.y = ex2_approx(y.y);
              acc = fadd2(acc, y);
              pk[8 * h + u] = F8 ? pack_f16x2(y.x, y.y) : pack_bf16x2(y.x, y.y);
            }
            l = fmaf(acc.x + acc.y, inv, l);
          }
          tmem_st16(S_row + c * 16, pk);
          if (c == 1) {
            // The accumulator: its last product was issued before this tile's S, which is complete.
            if (j > (alt ? w : 0) && __any_sync(kAll, resc)) {
              const uint32_t O_row = tmem + 256 + w * 128 + lane_off;
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 16) {
                uint32_t o[16];
                tmem_ld16(O_row + c0, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st16(O_row + c0, o);
              }
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(smem_u32(&bar_half[w]));
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&bar_p[w]));
      }
      if (!ok) break;
      // ---- the unit's part ends
      // The second warpgroup's statistics go through two columns behind its last weights, on the same
      // lanes.
      const bool other = alt && q.T > 1;
      float m1 = -INFINITY, l1 = 0.f;
      if (other && w == 1) {
        tmem_st2(S_row + 126, __float_as_uint(m_ref), __float_as_uint(l));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&bar_ml));
      } else if (other) {
        ok = wait_for(smem_u32(&bar_ml), odd_ml, abort_flag);
        if (!ok) break;
        odd_ml ^= 1;
        tc_fence_after();
        uint32_t a, b2;
        tmem_ld2(tmem + 128 + lane_off + 126, a, b2);
        tmem_ld_wait();
        tc_fence_before();
        m1 = __uint_as_float(a);
        l1 = __uint_as_float(b2);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_q_empty));
      // the next part
      Ring<kParts> here = pslot;
      pslot.next();
      const bool again = next_part() && ask(s_part[pslot.at]);
      if (alt && w == 1) {
        if (other) {
          ok = wait_for(smem_u32(&bar_o[1]), odd_o, abort_flag);
          if (!ok) break;
          odd_o ^= 1;
        }
      } else {
        ok = wait_for(smem_u32(&bar_o[w]), odd_o, abort_flag);
        odd_o ^= 1;
        if (ok && other) ok = wait_for(smem_u32(&bar_o[1]), odd_other, abort_flag);
        if (other || !alt) odd_other ^= 1;  // the second warpgroup had sums
        if (!ok) break;
        tc_fence_after();
        const bool final = q.whole_l && q.whole_r;
        const float top = fmaxf(m_ref, m1);
        float f0 = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - top);
        float f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - top);
        const float sum = l * f0 + l1 * f1;
        if (final) {
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          f0 *= inv;
          f1 *= inv;
        }
        const int rr = q.row0 + row, tok = in ? rr / p.group : 0;
        const int64_t at = (int64_t)(q.q0 + tok) * p.hq + q.g * p.group + (rr - tok * p.group);
        float* part = p.parts + (size_t)(2 * blockIdx.x + (q.whole_l ? 1 : 0)) * (C::kUnitRows * (D + 2));
        float* to32 = final ? static_cast<float*>(p.out) + at * D : part + row * 4;
        const int quad = final ? 4 : 4 * C::kUnitRows;  // from four columns to the next
        uint16_t* to16 = static_cast<uint16_t*>(p.out) + at * D;
#pragma unroll 1
        for (int c0 = 0; live && c0 < D; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tmem + 256 + w * 128 + lane_off + c0, o);
          tmem_ld_wait();
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * f0;
          if (other) {
            tmem_ld32(tmem + 384 + lane_off + c0, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(o[i]), f1, v[i]);
          }
          if (in) {
            if (final && p.out_bf16) {
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                *reinterpret_cast<uint4*>(to16 + c0 + i) =
                    make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                               pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(to32 + (c0 + i) / 4 * quad) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          }
          __syncwarp();
        }
        if (in) {
          if (!final)
            *reinterpret_cast<float2*>(part + C::kUnitRows * D + 2 * row) = make_float2(top, sum);
          else if (p.lse != nullptr)
            p.lse[at] = sum > 0.f ? (top - kBias + log2f(sum)) * kLn2 : -INFINITY;
        }
        tc_fence_before();
        if (!q.whole_l && q.whole_r && tid == 128) {  // tell the second launch where the unit began
          p.jobs[blockIdx.x] = make_int4(q.c0, q.rows, q.row0, q.g);
          p.job_q0[blockIdx.x] = q.q0;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_part_empty[here.at]));
      ok = again;
    }
    cp_async_wait_all();  // also where a wait ran out
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag && p.dev_status != nullptr) atomicOr(p.dev_status, kDevTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Parts c, c + step, .. c1 of a unit begun in CTA c0, of one row the columns [16 x, 16 x + 16): kBatch
// parts' loads are in flight.
template <int D, int kBatch>
__device__ __forceinline__ void join_parts(const Params& p, int c, int c0, int c1, int step, int row,
                                           bool in, int x, float& top, float& sum, float4 (&acc)[4]) {
  const int R = p.unit_rows;
  for (; c <= c1; c += kBatch * step) {
    float2 ml[kBatch];
    float4 v[kBatch][4];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int at = c + i * step;
      ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i][q] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (at <= c1 && in) {
        const float* part = p.parts + (size_t)(2 * at + (at == c0 ? 1 : 0)) * (R * (D + 2));
        ml[i] = *reinterpret_cast<const float2*>(part + R * D + 2 * row);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[i][q] = *reinterpret_cast<const float4*>(part + ((x * 4 + q) * (size_t)R + row) * 4);
      }
    }
    float n = top;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) n = fmaxf(n, ml[i].x);
    const float f = top == -INFINITY ? 0.f : ex2_approx(top - n);
    top = n;
    sum *= f;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      acc[q] = make_float4(acc[q].x * f, acc[q].y * f, acc[q].z * f, acc[q].w * f);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float fi = ml[i].x == -INFINITY ? 0.f : ex2_approx(ml[i].x - n);
      sum = fmaf(ml[i].y, fi, sum);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[q].x = fmaf(v[i][q].x, fi, acc[q].x);
        acc[q].y = fmaf(v[i][q].y, fi, acc[q].y);
        acc[q].z = fmaf(v[i][q].z, fi, acc[q].z);
        acc[q].w = fmaf(v[i][q].w, fi, acc[q].w);
      }
    }
  }
}

// Joins the parts of the units that CTA borders cut: block (c, y) for rows 32 y .. of the unit that
// ended in CTA c. A lane is a row, a warp 16 columns (the parts lie so that a warp reads whole lines), kBatch
// parts' loads are in flight, and each lane writes whole sectors. The parts are joined in the
// list's order.
template <int D>
__global__ void __launch_bounds__(2 * D) attn_tree_join_kernel(const Params p, float bias) {
  constexpr int kBatch = 4;
  const int c1 = blockIdx.x, warp = threadIdx.x >> 5, row = blockIdx.y * 32 + (threadIdx.x & 31);
  wait_for_prior_grids();  // the parts are written
  const int4 job = p.jobs[c1];
  const int q0 = p.job_q0[c1];
  if (job.x < 0 || row >= job.y) return;
  float top = -INFINITY, sum = 0.f;
  float4 acc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  join_parts<D, kBatch>(p, job.x, job.x, c1, 1, row, true, warp, top, sum, acc);
  const int rr = job.z + row, tok = rr / p.group;
  const int64_t at = (int64_t)(q0 + tok) * p.hq + job.w * p.group + (rr - tok * p.group);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int64_t to = at * D + warp * 16;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    acc[q] = make_float4(acc[q].x * inv, acc[q].y * inv, acc[q].z * inv, acc[q].w * inv);
  if (p.out_bf16) {
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + to);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      o[q] = make_uint4(pack_bf16x2(acc[2 * q].x, acc[2 * q].y), pack_bf16x2(acc[2 * q].z, acc[2 * q].w),
                        pack_bf16x2(acc[2 * q + 1].x, acc[2 * q + 1].y),
                        pack_bf16x2(acc[2 * q + 1].z, acc[2 * q + 1].w));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      reinterpret_cast<float4*>(static_cast<float*>(p.out) + to)[q] = acc[q];
  }
  if (p.lse != nullptr && warp == 0) p.lse[at] = sum > 0.f ? (top - bias + log2f(sum)) * kLn2 : -INFINITY;
}

// The same where units are few and have many parts each (kDeep at least on average, over the longest
// lists): block (u, y, z) for rows 32 y .., columns 16 z .. of unit u, whose parts follow from the
// lengths. A warp takes every kDeep-th part, kBatch at a time, and the warps' sums are joined in order
// through shared memory. One request of 2590 tokens and eight KV heads, eleven parts to a unit: 15.3 us
// with the kernel above (three rounds of loads, and blocks for every CTA), 13.4 with this one; 8192
// tokens and two KV heads, 76 parts to a unit: 29 and 15 us.
constexpr int kDeep = 8;
template <int D, bool kTwo>
__global__ void __launch_bounds__(kDeep * 32) attn_tree_join_deep_kernel(const Params p, float bias) {
  using C = Cfg<true, D, kTwo>;  // tiles and units are the same for either cache
  constexpr int kBatch = 4;
  __shared__ float2 s_ml[kDeep][32];
  __shared__ float s_acc[kDeep][32][17];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = (p.max_q * p.group + C::kUnitRows - 1) / C::kUnitRows;  // of rows, a unit each
  const int rt = blockIdx.x % blocks, g = blockIdx.x / blocks % p.hkv, b = blockIdx.x / blocks / p.hkv;
  wait_for_prior_grids();  // the parts are written
  uint32_t bad = 0;
  Req r;
  r.n = r.nt = r.rt = r.q0 = 0;
  if (lane < p.batch) r = load_req<C::kTK>(p, lane, &bad);
  const int v = places_of<C::kQTiles>(p, r), incl = warp_scan(v, lane);
  const int n = __shfl_sync(kAll, r.n, b), nt = __shfl_sync(kAll, r.nt, b),
            rts = __shfl_sync(kAll, r.rt, b), q0 = __shfl_sync(kAll, r.q0, b),
            places = __shfl_sync(kAll, v, b), before = __shfl_sync(kAll, incl, b) - places;
  if (rt >= rts) return;
  const int weight = rt == rts - 1 ? last_weight(p, n, C::kUnitRows) : C::kQTiles;
  const int begin = before + places / p.hkv * g + rt * (nt * C::kQTiles + kEndTiles);
  const Runs cut(__shfl_sync(kAll, incl, 31), p.ctas);
  const int c0 = cut.cta_of(begin), c1 = cut.cta_of(begin + weight * (nt - 1));
  const int row0 = blockIdx.y * 32, rows = min(n * p.group - rt * C::kUnitRows, C::kUnitRows);
  if (c0 == c1 || row0 >= rows) return;  // the same for the block
  const int row = row0 + lane;
  float top = -INFINITY, sum = 0.f;
  float4 acc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  join_parts<D, kBatch>(p, c0 + warp, c0, c1, kDeep, row, row < rows, blockIdx.z, top, sum, acc);
  s_ml[warp][lane] = make_float2(top, sum);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float* to = &s_acc[warp][lane][4 * q];
    to[0] = acc[q].x;
    to[1] = acc[q].y;
    to[2] = acc[q].z;
    to[3] = acc[q].w;
  }
  __syncthreads();
  // eight lanes write a row's 16 columns
  const int at_row = threadIdx.x >> 3, col = (threadIdx.x & 7) * 2;
  if (row0 + at_row >= rows) return;
  float m = -INFINITY, l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
  for (int w = 0; w < kDeep; ++w) m = fmaxf(m, s_ml[w][at_row].x);
#pragma unroll
  for (int w = 0; w < kDeep; ++w) {
    const float2 ml = s_ml[w][at_row];
    const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
    l = fmaf(ml.y, f, l);
    x = fmaf(s_acc[w][at_row][col], f, x);
    y = fmaf(s_acc[w][at_row][col + 1], f, y);
  }
  const int rr = rt * C::kUnitRows + row0 + at_row, tok = rr / p.group;
  const int64_t at = (int64_t)(q0 + tok) * p.hq + g * p.group + (rr - tok * p.group);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t to = at * D + blockIdx.z * 16 + col;
  if (p.out_bf16)
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + to) = pack_bf16x2(x * inv, y * inv);
  else
    *reinterpret_cast<float2*>(static_cast<float*>(p.out) + to) = make_float2(x * inv, y * inv);
  if (p.lse != nullptr && blockIdx.z == 0 && col == 0)
    p.lse[at] = l > 0.f ? (m - bias + log2f(l)) * kLn2 : -INFINITY;
}

// Rows of a unit: one q tile of 128, or two where a request may have more rows of one KV head.
int rows_of(int max_q, int group) { return (int64_t)max_q * group <= kRows ? kRows : 2 * kRows; }
size_t job_bytes(size_t ctas) {
  return (ctas * (sizeof(int4) + sizeof(int)) + 255) / 256 * 256;
}

template <bool F8, int D, bool kTwo>
cudaError_t launch(const AttnDecodeArgs& a, int dev, int sms, int* drv_err, cudaStream_t stream) {
  using C = Cfg<F8, D, kTwo>;
  Params p;
  p.q = static_cast<const uint16_t*>(a.q);
  p.cu_q = a.cu_q;
  p.mask = a.tree_mask;
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
  p.ctas = sms;
  p.unit_rows = C::kUnitRows;
  p.jobs = static_cast<int4*>(a.workspace);
  p.job_q0 = reinterpret_cast<int*>(p.jobs + p.ctas);
  p.parts =
      reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + job_bytes((size_t)p.ctas));
  CUtensorMap mk, mv;
  auto make = [&](CUtensorMap* m, void* base) -> bool {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.page_size, (uint64_t)a.num_pages * a.hkv};
    const uint64_t strides[2] = {(uint64_t)C::kRowBytes, (uint64_t)C::kRowBytes * a.page_size};
    const uint32_t box[3] = {(uint32_t)(F8 ? D : 64),
                             (uint32_t)a.page_size, 1};  // pages have 128 tokens at most
    const CUresult e = encode_tensor_map(
        m, F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims,
        strides, box, C::kPanelBytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
    if (e != CUDA_SUCCESS) *drv_err = (int)e;
    return e == CUDA_SUCCESS;
  };
  if (!make(&mk, const_cast<void*>(a.k_cache)) || !make(&mv, const_cast<void*>(a.v_cache)))
    return cudaErrorInvalidValue;
  auto kernel = attn_tree_kernel<F8, D, kTwo>;
  // The registers that move between the warps must be those that the block is launched with.
  static std::atomic<int> known{0};
  int regs = 0;
  cudaError_t e = ask_once(known, &regs, [&](int* n) {
    cudaFuncAttributes f;
    const cudaError_t err = cudaFuncGetAttributes(&f, kernel);
    if (err == cudaSuccess) *n = f.numRegs;
    return err;
  });
  if (e != cudaSuccess) return e;
  if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  // The kernel's shared-memory limit is set once per device (bit i: device i), not per call. A
  // launch that fails has it set again.
  static std::atomic<uint64_t> set{0};
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  e = launch_ahead(kernel, dim3(p.ctas), kThreads, C::kSmemBytes, stream, mk, mv, p);
  if (e != cudaSuccess) {
    set.fetch_and(~bit, std::memory_order_relaxed);
    return e;
  }
  const float bias = F8 ? 11.f : 0.f;
  const int64_t rows = (int64_t)p.max_q * p.group;
  const int64_t units = (rows + C::kUnitRows - 1) / C::kUnitRows * p.hkv * p.batch;
  const unsigned blocks = (unsigned)((std::min<int64_t>(rows, C::kUnitRows) + 31) / 32);
  if (units * kDeep <= p.ctas && p.batch <= 32)
    return launch_ahead(attn_tree_join_deep_kernel<D, kTwo>, dim3((unsigned)units, blocks, D / 16),
                        kDeep * 32, 0, stream, p, bias);
  return launch_ahead(attn_tree_join_kernel<D>, dim3(p.ctas, blocks), 2 * D, 0, stream, p, bias);
}

template <bool F8, int D>
cudaError_t launch_rows(const AttnDecodeArgs& a, int dev, int sms, int* drv_err,
                        cudaStream_t stream) {
  return rows_of(a.max_q, a.hq / a.hkv) == kRows ? launch<F8, D, false>(a, dev, sms, drv_err, stream)
                                                 : launch<F8, D, true>(a, dev, sms, drv_err, stream);
}

}  // namespace

size_t attn_tree_workspace_bytes(int max_q, int hq, int hkv, int d, int sms) {
  const size_t ctas = (size_t)sms, rows = rows_of(max_q, hq / hkv);
  return job_bytes(ctas) + ctas * 2 * rows * (d + 2) * sizeof(float);
}

cudaError_t launch_attn_tree(const AttnDecodeArgs& a, int* drv_err, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (a.d == 64)
    return a.f8 ? launch_rows<true, 64>(a, dev, sms, drv_err, stream)
                : launch_rows<false, 64>(a, dev, sms, drv_err, stream);
  if (a.d == 128)
    return a.f8 ? launch_rows<true, 128>(a, dev, sms, drv_err, stream)
                : launch_rows<false, 128>(a, dev, sms, drv_err, stream);
  return cudaErrorInvalidValue;
}

}  // namespace tts
