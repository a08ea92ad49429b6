// Dense attention forward (non-causal vision and varlen causal GQA prefill).
//
// What it computes: for every query row, softmax(scale * q K^T) V over the
// visible keys, plus lse = ln sum exp(scale * q k) -- the S-gemm / softmax /
// PV-gemm pieces of "DeepSeek V4.1 上 4×RTX 3090" (section 三), over the
// cu_seqlens batches of "从 SGLang Kernel源码到 GPU Trace" (section 2.2, keys past
// a sequence's length skipped as in section 3.2), FP32 statistics and FP32
// accumulation as in "AMD MI250部署DeepSeek-V4-Flash" (3.1, 4.1), causal mask
// as -inf (3.3), and the online-softmax merge of "推理引擎的蝴蝶效应" (进一步探索,
// equations 1-2) applied tile after tile in a fixed order.
//
// How: one persistent CTA per SM takes work items -- (sequence, 256-row query
// pair, head), heaviest first -- from a global counter in the caller's workspace:
//   warp 0        TMA producer: picks the items, then per item K/V 128-row tiles
//                 into a ring and the two Q tiles (the next item's loads overlap
//                 the current item's last tiles and epilogue)
//   warp 1        TMEM allocator + tcgen05 MMA issuer (the whole warp runs the
//                 issue loop converged; one elected lane issues)
//   warps 4..7    softmax warpgroup 0 (query rows 0..127 of the pair)
//   warps 8..11   softmax warpgroup 1 (query rows 128..255)
// TMEM (512 columns): S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D).
// S = Q K^T lands in TMEM; each softmax thread owns one row (TMEM lane), keeps
// the running max / sum in fp32 registers, writes P as bf16 pairs over the first
// 64 columns of its S region, and the MMA warp issues O += P V with P read
// straight from TMEM. The two warpgroups ping-pong so the tensor core works
// on one tile's MMAs while the other tile's softmax runs.
// The running max is only moved (and O rescaled) when it grows by more than
// 2^8 in the exp2 domain; otherwise P uses the older max, which bounds P by
// 256 and is exact in real arithmetic (the final O / l cancels the offset).
// No S or P matrix ever touches global memory, so there is no piece buffer
// to index (the q0*N overflow of the vision write-up cannot happen here).
//
// With a sliding window (kWin, causal): row i at position P = i + Lk - Lq sees keys
// (P - window, P] and the first `sinks`, so an item streams only the tiles that one of its
// rows sees: the sinks' tiles, then the window's. The work per row is then 4 d min(P + 1,
// window + sinks) whatever the prompt's length. Rows of a last tile behind the sequence's
// end (another sequence's, or padding), and keys that no row of the sequence sees (between the
// first tokens and the first row's window), are cleared in V before the product, so that what
// they hold cannot reach a row through a weight of zero.
// What differs from the kernel without a window, because its items are short: the producer hands the
// decoded item on; registers move to the softmax warps; the products with a tile's first 64
// weights start while the others are computed; rows leave by TMA stores; and the code is kept
// small, since an item runs once through all of it and what the instruction cache misses is a
// fifth of the softmax warps' time.
// Measured: 16,000 tokens, window 4096, 128 sinks, 16 / 4 heads of 128: 302 to 324 us, 1.48 to
// 1.59 PFLOP/s over visible pairs (0.78 to 0.83 of the measured bf16 rate; 1.27 us per pair of
// tiles, the tensor core's rate, and 3 us per item; 286 in a graph that repeats it on the same
// data); four prompts of 827 to 3212 tokens, window 1024, 32 / 8 heads: 100 to 103 us, 0.94
// PFLOP/s (ten tiles for the keys of eight: the sinks' tile and two at the window's ends, whose
// masks add to each; 6.4 items per CTA at 3 us each); 700 tokens, window 256, 8 / 2 heads of 64:
// 9.7 to 10.7 us, launch, five tiles' chain of 1.3 us each, and the rows' store. Smaller heads
// keep the softmax work per score and have fewer products beside it: three prompts of 3000 to 8000
// tokens, window 1024, 32 / 8 heads of 64, 80 and 128: 186, 205 and 221 us.
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tts {
namespace {

constexpr int kAttnThreads = 384;
constexpr int kBlockM = 128;  // query rows per softmax warpgroup
constexpr int kBlockN = 128;  // keys per K/V tile

// Instruction descriptor for kind::f8f6f4 with e4m3 A and B (format code 0), fp32 D,
// both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | (0u << 7) | (0u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// D[tmem] (+)= A[smem] * B[smem], e4m3 operands, from the elected lane of a converged warp.
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

// F8: q and k are e4m3 (one byte per value) and S = Q K^T runs as kind::f8f6f4 MMAs;
// V, P and O stay bf16 / fp32. Built for D = 128 only.
template <int D, bool F8 = false>
struct AttnCfg {
  static constexpr int kQKCols = F8 ? 128 : 64;  // q / k values per 128-byte row
  static constexpr int kMainBoxes = D / kQKCols;  // SW128 boxes of q / k
  static constexpr int kTail = F8 ? 0 : D % 64;   // 0 or 16 (SW32 box)
  static constexpr int kBoxBytes = kBlockN * 128;  // one SW128 box of 128 rows
  static constexpr int kTailBytes = kBlockN * 32;  // one SW32 box of 128 rows
  static constexpr int kTileBytes = kMainBoxes * kBoxBytes + (kTail ? kTailBytes : 0);
  // V for d=80 is loaded as three 32-column SW64 boxes (d 80..95 zero-filled by the
  // tensor map's bounds) so that one N=96 MMA per K step covers it; d=64/128 reuse the
  // K/Q layout.
  static constexpr int kVBoxes = kTail ? 3 : D / 64;
  static constexpr int kVBoxBytes = kTail ? kBlockN * 64 : kBoxBytes;
  static constexpr int kVTileBytes = kVBoxes * kVBoxBytes;
  static constexpr int kPvN = kTail ? 96 : D;
  static constexpr int kStages = (D <= 80 || F8) ? 3 : 2;
  static constexpr int kStageBytes = 8 * 4096;  // output staging, 4 KB per softmax warp
  static constexpr int kSmemBytes =
      (2 + kStages) * kTileBytes + kStages * kVTileBytes + kStageBytes + 1024;
  static_assert(kTail == 0 || kTail == 16, "head_dim must be 64, 80 or 128");
  static_assert(!F8 || D == 128, "the e4m3 q / k path is built for head_dim 128");
};

struct AttnMaps {
  CUtensorMap q, k, v;           // SW128 boxes {64, 1, 128} (q / k e4m3: {128, 1, 128})
  CUtensorMap q_t, k_t;          // SW32 boxes {16, 1, 128} for the d=64..79 tail
  CUtensorMap v_t;               // d=80: SW64 boxes {32, 1, 128} for all of V
};
struct WindowMaps : AttnMaps {
  CUtensorMap o;  // out, 128-byte boxes of 32 rows: {64 bf16 or 32 fp32, 1, 32}
};
template <bool kWin>
using MapsFor = std::conditional_t<kWin, WindowMaps, AttnMaps>;

struct AttnParams {
  const int32_t* cu_q;
  const int32_t* cu_k;
  uint32_t* work_counter;  // items handed out so far (zeroed before the launch)
  int n_items;
  float* out;
  float* lse;
  uint32_t* dev_status;
  int64_t total_q, total_k;
  int batch, max_seqlen_q, max_seqlen_k, hq, hkv, causal, pairs_max;
  float scale, scale_log2;
  const float* q_scale;  // e4m3 path: [total_q, hq] per (token, head)
  const float* k_scale;  // e4m3 path: [hkv] per KV head
};
struct WindowParams : AttnParams {
  int window, sinks;  // keys up to a row's own, first keys that stay visible
  int out_bf16;       // out is bf16
  // What the two query tiles of an item are. kHeads: two heads of a KV group on the same 128
  // rows (an even group): both see the same keys, where two tiles of consecutive rows (kRows,
  // an odd group) stream one tile more than each needs (ragged batch, window 1024: 213 -> 116
  // us, with the masks as words). kSolo: one tile alone, where all of them fit the GPU at once: a
  // tile's chain is shorter without a second tile's between its steps.
  enum Pairing : int { kRows, kHeads, kSolo };
  int pairing;
};
template <bool kWin>
using ParamsFor = std::conditional_t<kWin, WindowParams, AttnParams>;

// kWin: registers move from the warpgroup of the issuing warps to the two softmax warpgroups,
// which hold 128 scores and the masks. 128 x 80 + 256 x 208 = 63488 of the
// 384 x 168 = 64512 that the block is launched with.
constexpr int kIssueRegs = 80, kSoftmaxRegs = 208;
// The sum must not pass what the block was launched with, or the taking warps would wait for ever;
// the launch looks at the compiled kernel's registers before its first call.
constexpr int kLaunchRegs = (128 * kIssueRegs + 256 * kSoftmaxRegs + kAttnThreads - 1) / kAttnThreads;
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Load one 128-row tile (all boxes) of a [tokens, heads, D] tensor (F8: of e4m3 q / k).
template <int D, bool F8 = false>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* main,
                                          const CUtensorMap* tail, uint32_t bar, int head,
                                          int token) {
  using C = AttnCfg<D, F8>;
#pragma unroll
  for (int b = 0; b < C::kMainBoxes; ++b)
    tma_load_3d(dst + b * C::kBoxBytes, main, bar, b * C::kQKCols, head, token);
  if constexpr (C::kTail != 0)
    tma_load_3d(dst + C::kMainBoxes * C::kBoxBytes, tail, bar, C::kMainBoxes * 64, head, token);
}

// S[tmem] = Q[smem] K[smem]^T over the D-deep contraction. q_d / k_d are the
// descriptors of the tiles' first box; every other K step is a constant offset
// (the 14-bit start-address field never carries: shared addresses are < 256 KB).
// e: the elected lane of the converged issuing warp.
// F8: e4m3 x e4m3 -> fp32, K = 32 per MMA, so the same 32-byte steps cover the row.
template <int D, bool F8 = false>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint64_t q_d, uint64_t k_d,
                                         uint64_t q_tail_d, uint64_t k_tail_d, uint32_t e) {
  using C = AttnCfg<D, F8>;
  constexpr uint32_t idesc =
      F8 ? idesc_e4m3_f32(128, kBlockN) : idesc_bf16_f32(128, kBlockN, 0, 0);
#pragma unroll
  for (int ks = 0; ks < C::kMainBoxes * 4; ++ks) {
    const uint32_t off = ((ks / 4) * C::kBoxBytes + (ks % 4) * 32) >> 4;
    if constexpr (F8)
      mma_ss_f8_elect(d_tmem, q_d + off, k_d + off, idesc, ks > 0, e);
    else
      mma_ss_elect(d_tmem, q_d + off, k_d + off, idesc, ks > 0, e);
  }
  if constexpr (C::kTail != 0) mma_ss_elect(d_tmem, q_tail_d, k_tail_d, idesc, 1, e);
}

// O[tmem] (+)= P[tmem] V[smem]; V is MN-major (d contiguous). v_d describes the
// first V box (SW128 boxes for d=64/128, SW64 boxes for d=80).
// Keys [16 kFrom, 16 kTo) of the tile.
template <int D, int kFrom = 0, int kTo = kBlockN / 16>
__device__ __forceinline__ void issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint64_t v_d,
                                         uint32_t accumulate, uint32_t e) {
  using C = AttnCfg<D>;
  constexpr uint32_t idesc = idesc_bf16_f32(128, C::kPvN, 0, 1);
  constexpr uint32_t kStep = C::kTail ? 16 * 64 : 16 * 128;  // 16 key rows of one box
#pragma unroll
  for (int ks = kFrom; ks < kTo; ++ks)
    mma_ts_elect(o_tmem, p_tmem + ks * 8, v_d + ((ks * kStep) >> 4), idesc,
                 (ks > 0) ? 1u : accumulate, e);
}


// exp2_pack_sum with the four partial sums carried from part to part, and their total.
template <int N>
__device__ __forceinline__ void exp2_pack_acc(uint32_t* sr, float c, float nmc, float2 (&acc)[4]) {
  const float* s = reinterpret_cast<const float*>(sr);
  const float2 c2 = make_float2(c, c), nm2 = make_float2(nmc, nmc);
#pragma unroll
  for (int k0 = 0; k0 < N / 2; k0 += 8) {
    float2 x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      x[u] = ffma2(make_float2(s[2 * (k0 + u)], s[2 * (k0 + u) + 1]), c2, nm2);
      x[u].x = ex2_approx(x[u].x);
      x[u].y = ex2_approx(x[u].y);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      acc[u & 3] = fadd2(acc[u & 3], x[u]);
      sr[k0 + u] = pack_bf16x2(x[u].x, x[u].y);
    }
  }
}
__device__ __forceinline__ float sum_of(const float2 (&acc)[4]) {
  const float2 a = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
  return a.x + a.y;
}

// One work item = (256-row query pair, sequence, head); `it` enumerates them with
// the heaviest (latest, causal) pairs of every sequence first. Every role decodes
// an item the same way. Returns false for items with nothing to compute and for
// sequences whose cu_seqlens entries are invalid.
struct Item {
  int64_t q_start, k_start, Lq, Lk, q_lo;
  int h, g, n_tiles;  // n_tiles: K/V tiles streamed = max(n0, n1)
  int n0, n1;         // tiles each warpgroup needs (0: no rows, or no visible key)
  int n_sink, win0;   // kWin: streamed tiles are [0, n_sink), then win0, win0 + 1, ...
  int dh, dr;         // kWin: head and row of the second warpgroup's tile, from the first's
};
// Key tile that an item streams as its j-th.
template <bool kWin>
__device__ __forceinline__ int key_tile(const Item& w, int j) {
  if constexpr (kWin) return j < w.n_sink ? j : w.win0 + (j - w.n_sink);
  return j;
}
template <bool kWin>
__device__ __forceinline__ bool decode_item(const ParamsFor<kWin>& p, int it, Item& w, bool* bad) {
  int heads = p.hq;
  if constexpr (kWin) heads = p.pairing == WindowParams::kHeads ? p.hq / 2 : p.hq;
  int h = it % heads;
  const int t = it / heads;
  const int b = t % p.batch;
  const int pr = p.pairs_max - 1 - t / p.batch;
  const int64_t q_start = p.cu_q[b], k_start = p.cu_k[b];
  const int64_t q_end = p.cu_q[b + 1], k_end = p.cu_k[b + 1];
  const int64_t Lq = q_end - q_start, Lk = k_end - k_start;
  *bad = false;
  if (q_start < 0 || k_start < 0 || Lq < 0 || Lk < 0 || q_end > p.total_q || k_end > p.total_k ||
      Lq > p.max_seqlen_q || Lk > p.max_seqlen_k) {
    *bad = (pr == 0 && h == 0);  // report each bad sequence once
    return false;
  }
  // First query row of the pair (within the sequence). With an odd number of 128-row
  // query tiles the pairs start one tile early, so the tile without a partner is tile 0
  // (the cheapest under a causal mask: one key tile) and the first warpgroup of pair 0
  // has no rows.
  const int64_t n_qt = (Lq + kBlockM - 1) / kBlockM;
  int64_t q_lo = (int64_t)pr * 2 * kBlockM - ((n_qt & 1) ? kBlockM : 0);
  int64_t row1 = kBlockM;  // the second warpgroup's rows, from the first's
  if constexpr (kWin) {
    w.dh = 0;
    w.dr = kBlockM;
    if (p.pairing != WindowParams::kRows) q_lo = (int64_t)pr * kBlockM;
    if (p.pairing == WindowParams::kHeads) {
      h *= 2;
      w.dh = 1;
      w.dr = 0;
      row1 = 0;
    }
  }
  if (q_lo >= Lq) return false;
  // Keys each warpgroup's rows can see: all of them, or (causal) up to its last row's
  // diagonal; none for a warpgroup without rows (the odd last tile of a sequence).
  auto keys_for = [&](int64_t r_first, int64_t r_end) -> int64_t {
    if (r_first >= Lq || r_end <= 0) return 0;
    if (!p.causal) return Lk;
    const int64_t lim = (r_end < Lq ? r_end : Lq) - 1 + (Lk - Lq) + 1;
    return lim < 0 ? 0 : (lim < Lk ? lim : Lk);
  };
  const int64_t kv_end0 = keys_for(q_lo, q_lo + kBlockM);
  int64_t kv_end1 = keys_for(q_lo + row1, q_lo + row1 + kBlockM);
  if constexpr (kWin) {
    if (p.pairing == WindowParams::kSolo) {
      kv_end1 = row1 = 0;
      // the second warpgroup's rows are all behind the sequence: the next ones are another item's
      w.dr = (int)n_qt * kBlockM;
    }
  }
  const int64_t kv_end = kv_end0 > kv_end1 ? kv_end0 : kv_end1;
  w.q_start = q_start;
  w.k_start = k_start;
  w.Lq = Lq;
  w.Lk = Lk;
  w.q_lo = q_lo;
  w.h = h;
  w.g = h / (p.hq / p.hkv);
  w.n_tiles = (int)((kv_end + kBlockN - 1) / kBlockN);
  w.n0 = (int)((kv_end0 + kBlockN - 1) / kBlockN);
  w.n1 = (int)((kv_end1 + kBlockN - 1) / kBlockN);
  if constexpr (kWin) {
    // First key inside the window of the first row that sees any (a later row's starts later).
    const int64_t off = Lk - Lq;
    const int64_t row = kv_end0 > 0 ? (q_lo > 0 ? q_lo : 0) : q_lo + row1;
    const int64_t lo = row + off + 1 - p.window;
    // Last row's window: the first keys that no window of the item holds are kept apart.
    const int64_t lo1 = q_lo + row1 + kBlockM - 1 + off + 1 - p.window;
    w.win0 = lo > 0 ? (int)(lo / kBlockN) : 0;
    const int64_t sinks = p.sinks < lo1 ? p.sinks : lo1;  // more are inside every window
    const int64_t ns = sinks > 0 ? (sinks + kBlockN - 1) / kBlockN : 0;
    w.n_sink = (int)(ns < w.win0 ? ns : w.win0);
    const int skip = w.win0 - w.n_sink;  // tiles in between that no row sees
    w.n_tiles = w.n_tiles > 0 ? w.n_tiles - skip : 0;
    w.n0 = w.n0 > 0 ? w.n0 - skip : 0;
    w.n1 = w.n1 > 0 ? w.n1 - skip : 0;
  }
  return true;
}

// Waits of the kernel. kWin: the same bounded wait in half the instructions (32-bit nanoseconds,
// the status set once at the end): its code competes with the tiles' for the instruction cache
// (ragged prompts, window 1024: 104 -> 101 us; window 128: 67 -> 63). The issuing warp looks
// without suspending first (288 us; 310 without, 16,000 tokens).
template <bool kWin>
__device__ __forceinline__ bool thread_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                            uint32_t* status) {
  if constexpr (!kWin) return mbar_wait(bar, parity, abort, status);
  uint32_t since = 0;
  while (!mbar_test(bar, parity)) {
    if (*abort) return false;
    uint32_t now;
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(now));
    if (since == 0) since = now | 1u;
    const int waited = (int)(now - since);  // -1 to what one suspension and the limit add up to
    if (waited > (int)kWaitLimitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
template <bool kWin>
__device__ __forceinline__ bool all_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                         uint32_t* status) {
  if constexpr (!kWin) return warp_wait(bar, parity, abort, status);
  const bool ok = mbar_peek(bar, parity) || thread_wait<kWin>(bar, parity, abort, status);
  return __all_sync(0xFFFFFFFFu, ok);
}

// Persistent: one CTA per SM takes items from a global counter until none are left (kWin: its one
// item where there are no more items than CTAs).
// Per CTA, items flow through a two-slot ring (producer -> MMA warp + softmax warps);
// barrier phases run on counters that continue across items: gt = K/V tiles so far
// (ring slots, S / P phases), nq = items with at least one tile (Q, O phases).
template <int D, bool F8 = false, bool kWin = false>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_fwd_kernel(const __grid_constant__ MapsFor<kWin> maps, const ParamsFor<kWin> p) {
  using C = AttnCfg<D, F8>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  // bar_k / bar_v: K and V of a tile landed. With three stages (d <= 80) the V load
  // has time to land before the S MMA that first needs the tile, so both share bar_k
  // and the MMA warp waits once per tile; with two stages (d = 128) V gets its own
  // barrier so S(j+1) does not wait for V(j+1), and K's slot is released (bar_k_empty)
  // as soon as both S MMAs of its tile are done, a PV pair before V's slot
  // (bar_kv_empty), so the next K load starts that much earlier.
  constexpr bool kOneKV = NS >= 3;
  __shared__ __align__(8) uint64_t bar_item_full[2], bar_item_empty[2], bar_q[2], bar_q_empty[2],
      bar_k[NS], bar_v[NS], bar_k_empty[NS], bar_kv_empty[NS], bar_s[2], bar_p[2], bar_o[2],
      bar_drain;
  __shared__ int s_item[2];
  __shared__ Item s_work[2];  // kWin: the decoded items
  __shared__ __align__(8) uint64_t bar_half[2];  // kWin: the weights of a tile's first 64 keys
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t s_base = smem_u32(smem);
  const uint32_t sQ[2] = {s_base, s_base + C::kTileBytes};
  auto sK = [&](int st) { return s_base + (2 + st) * C::kTileBytes; };
  auto sV = [&](int st) {
    return s_base + (2 + NS) * C::kTileBytes + st * C::kVTileBytes;
  };
  // Output staging: 4 KB per softmax warp, after the K/V ring.
  uint8_t* stage_base = smem + (2 + NS) * C::kTileBytes + NS * C::kVTileBytes;

  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_item_full[i]), 1);
      mbar_init(smem_u32(&bar_item_empty[i]), 1 + 8);  // MMA warp + 8 softmax warps
      mbar_init(smem_u32(&bar_q[i]), 1);
      mbar_init(smem_u32(&bar_q_empty[i]), 1);
      mbar_init(smem_u32(&bar_s[i]), 1);
      mbar_init(smem_u32(&bar_p[i]), kBlockM);
      mbar_init(smem_u32(&bar_o[i]), 1);
      if constexpr (kWin) mbar_init(smem_u32(&bar_half[i]), kBlockM);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&bar_k[i]), 1);
      mbar_init(smem_u32(&bar_v[i]), 1);
      mbar_init(smem_u32(&bar_k_empty[i]), 1);
      mbar_init(smem_u32(&bar_kv_empty[i]), 1);
    }
    mbar_init(smem_u32(&bar_drain), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  volatile int* item_slot = s_item;
  if constexpr (kWin) {
    if (tid == 64) {  // on their way while the first item is found
      prefetch_tmap(&maps.q);
      prefetch_tmap(&maps.k);
      prefetch_tmap(&maps.v);
      prefetch_tmap(&maps.o);
    }
    wait_for_prior_grids();
  }

  if (warp < 4) {
  if constexpr (kWin) give_registers<kIssueRegs>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      if constexpr (!kWin) {
        prefetch_tmap(&maps.q);
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
      }
      int ni = 0, nq = 0, gt = 0;
      bool own = true;  // without a counter: this CTA's item is still to come
      int last_k[NS], last_v[NS];  // latest tile armed on each ring slot (-1: none)
      for (int i = 0; i < NS; ++i) last_k[i] = last_v[i] = -1;
      int q_armed[2] = {0, 0};  // per Q tile: items whose Q copy was started
      // Start the K (and V) copies of ring tile gj = item tile j.
      auto load_k = [&](int gj, const Item& w, int j) -> bool {
        const int st = gj % NS;
        const uint32_t empty_ph = ((gj / NS) - 1) & 1;
        if (gj >= NS && !thread_wait<kWin>(smem_u32(kOneKV ? &bar_kv_empty[st] : &bar_k_empty[st]),
                                   empty_ph, abort_flag, p.dev_status))
          return false;
        const int tok = (int)(w.k_start + (int64_t)key_tile<kWin>(w, j) * kBlockN);
        const uint32_t bk = smem_u32(&bar_k[st]);
        mbar_arrive_expect_tx(bk, kOneKV ? C::kTileBytes + C::kVTileBytes : C::kTileBytes);
        load_tile<D, F8>(sK(st), &maps.k, &maps.k_t, bk, w.g, tok);
        last_k[st] = gj;
        return true;
      };
      auto load_v = [&](int gj, const Item& w, int j) -> bool {
        const int st = gj % NS;
        const uint32_t bv = smem_u32(kOneKV ? &bar_k[st] : &bar_v[st]);
        if (!kOneKV) {
          if (gj >= NS && !thread_wait<kWin>(smem_u32(&bar_kv_empty[st]), ((gj / NS) - 1) & 1, abort_flag,
                                     p.dev_status))
            return false;
          mbar_arrive_expect_tx(bv, C::kVTileBytes);
        }
        const int tok = (int)(w.k_start + (int64_t)key_tile<kWin>(w, j) * kBlockN);
        if constexpr (C::kTail != 0) {
#pragma unroll
          for (int b = 0; b < C::kVBoxes; ++b)
            tma_load_3d(sV(st) + b * C::kVBoxBytes, &maps.v_t, bv, b * 32, w.g, tok);
        } else {
          load_tile<D>(sV(st), &maps.v, &maps.v, bv, w.g, tok);
        }
        last_v[st] = gj;
        return true;
      };
      bool ok = true;
      while (ok) {
        Item w;
        int it;
        for (;;) {  // next item with work (bad sequences are reported here, once)
          if (kWin && p.work_counter == nullptr) {
            it = own ? (int)blockIdx.x : p.n_items;
            own = false;
          } else {
            it = (int)atomicAdd(p.work_counter, 1u);
          }
          if (it >= p.n_items) {
            it = -1;
            break;
          }
          bool bad;
          if (decode_item<kWin>(p, it, w, &bad)) break;
          if (bad && p.dev_status) atomicOr(p.dev_status, kDevBadArg);
        }
        const int slot = ni & 1;
        if (ni >= 2 &&
            !thread_wait<kWin>(smem_u32(&bar_item_empty[slot]), ((ni >> 1) - 1) & 1, abort_flag,
                       p.dev_status))
          break;
        item_slot[slot] = it;
        if constexpr (kWin) s_work[slot] = w;
        mbar_arrive(smem_u32(&bar_item_full[slot]));  // release: the slot write is visible
        ++ni;
        if (it < 0) break;
        const int n = w.n_tiles;
        if (n == 0) continue;
        // The first ring tiles go first (their slots free up while the previous item
        // finishes); Q waits for the previous item's last S MMAs; the remaining tiles
        // need slots that this item's own MMAs free, so they come after Q.
        int pre = n < NS ? n : NS;
        // kWin, items of few tiles: the slot of the previous item's last tile is free only when
        // that item is done, its last S MMAs a tile earlier, so Q comes before the tile that
        // needs it (and first of all in a CTA's first item).
        if constexpr (kWin) pre = nq == 0 ? 0 : n < NS - 1 ? n : NS - 1;
        for (int j = 0; ok && j < pre; ++j) ok = load_k(gt + j, w, j) && load_v(gt + j, w, j);
        for (int wq = 0; ok && wq < 2; ++wq) {
          if (nq >= 1 && !thread_wait<kWin>(smem_u32(&bar_q_empty[wq]), (nq - 1) & 1, abort_flag,
                                    p.dev_status)) {
            ok = false;
            break;
          }
          const uint32_t bq = smem_u32(&bar_q[wq]);
          mbar_arrive_expect_tx(bq, C::kTileBytes);
          if constexpr (kWin)
            load_tile<D, F8>(sQ[wq], &maps.q, &maps.q_t, bq, w.h + wq * w.dh,
                             (int)(w.q_start + w.q_lo + wq * w.dr));
          else
            load_tile<D, F8>(sQ[wq], &maps.q, &maps.q_t, bq, w.h,
                       (int)(w.q_start + w.q_lo + wq * kBlockM));
          q_armed[wq] = nq + 1;
        }
        for (int j = pre; ok && j < n; ++j) ok = load_k(gt + j, w, j) && load_v(gt + j, w, j);
        gt += n;
        ++nq;
      }
      if (*abort_flag) {
        // Best-effort drain of copies still in flight before the CTA can exit: each
        // barrier's latest armed phase is the only one that can still be pending.
        for (int wq = 0; wq < 2; ++wq)
          if (q_armed[wq] > 0)
            mbar_wait(smem_u32(&bar_q[wq]), (q_armed[wq] - 1) & 1, nullptr, nullptr);
        for (int st = 0; st < NS; ++st) {
          if (last_k[st] >= 0)
            mbar_wait(smem_u32(&bar_k[st]), (last_k[st] / NS) & 1, nullptr, nullptr);
          if (!kOneKV && last_v[st] >= 0)
            mbar_wait(smem_u32(&bar_v[st]), (last_v[st] / NS) & 1, nullptr, nullptr);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t e = elect_one();
    const uint32_t S_t[2] = {tmem, tmem + 128};
    const uint32_t O_t[2] = {tmem + 256, tmem + 384};
    constexpr uint32_t kTailOff = C::kMainBoxes * C::kBoxBytes;
    uint64_t qd[2], qtd[2], kd[NS], ktd[NS], vd[NS];
    for (int w = 0; w < 2; ++w) {
      qd[w] = smem_desc(sQ[w], 16, 1024, kSw128);
      qtd[w] = smem_desc(sQ[w] + kTailOff, 16, 256, kSw32);
    }
    for (int i = 0; i < NS; ++i) {
      kd[i] = smem_desc(sK(i), 16, 1024, kSw128);
      ktd[i] = smem_desc(sK(i) + kTailOff, 16, 256, kSw32);
      vd[i] = C::kTail ? smem_desc(sV(i), C::kVBoxBytes, 512, kSw64)
                       : smem_desc(sV(i), C::kBoxBytes, 1024, kSw128);
    }
    // gt: K/V tiles so far (ring phases); g0 / g1: tiles of each warpgroup so far (S and P
    // phases); nq: items with tiles (Q phases).
    int ni = 0, nq = 0, gt = 0, g0 = 0, g1 = 0;
    bool ok = true;
    // PV of tile j (ring stage st) of warpgroup w once its weights are there; kWin: the first 64
    // keys' products start while the weights of the others are still computed.
    auto pv = [&](int w, int st, int j, int tiles) -> bool {
      const uint32_t ph = (tiles + j) & 1;
      if constexpr (kWin) {
        if (!all_wait<kWin>(smem_u32(&bar_half[w]), ph, abort_flag, p.dev_status)) return false;
        tc_fence_after();
        issue_pv<D, 0, 4>(O_t[w], S_t[w], vd[st], j > 0, e);
      }
      if (!all_wait<kWin>(smem_u32(&bar_p[w]), ph, abort_flag, p.dev_status)) return false;
      tc_fence_after();
      issue_pv<D, kWin ? 4 : 0>(O_t[w], S_t[w], vd[st], j > 0, e);
      return true;
    };
    while (ok) {
      const int slot = ni & 1;
      if (!all_wait<kWin>(smem_u32(&bar_item_full[slot]), (ni >> 1) & 1, abort_flag, p.dev_status))
        break;
      const int it = item_slot[slot];
      Item w;
      if constexpr (kWin) w = s_work[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_item_empty[slot]));
      ++ni;
      if (it < 0) break;
      if constexpr (!kWin) {
        bool bad;
        decode_item<kWin>(p, it, w, &bad);
      }
      const int n = w.n_tiles, n0 = w.n0, n1 = w.n1;
      if (n == 0) continue;
      int tail_row = kBlockN;  // kWin: first row of the last tile that is behind the sequence
      // kWin: keys [sinks, hid_end) are hidden from every row of the sequence. Tiles up to last_hid
      // may hold some: the sinks' last one and the window's first.
      int64_t hid_end = 0;
      int last_hid = -1;
      if constexpr (kWin) {
        tail_row = (int)(w.Lk - (int64_t)key_tile<true>(w, n - 1) * kBlockN);
        hid_end = w.Lk - w.Lq + 1 - p.window;
        if (hid_end > p.sinks)
          last_hid = (int64_t)w.win0 * kBlockN < hid_end ? w.n_sink : w.n_sink - 1;
      }
      const int st0 = gt % NS;
      ok = all_wait<kWin>(smem_u32(&bar_q[0]), nq & 1, abort_flag, p.dev_status) &&
           all_wait<kWin>(smem_u32(&bar_k[st0]), (gt / NS) & 1, abort_flag, p.dev_status);
      if (!ok) break;
      tc_fence_after();
      if (n0 > 0) {
        issue_qk<D, F8>(S_t[0], qd[0], kd[st0], qtd[0], ktd[st0], e);
        mma_commit_elect(smem_u32(&bar_s[0]), e);
      }
      if (n0 <= 1) mma_commit_elect(smem_u32(&bar_q_empty[0]), e);
      ok = all_wait<kWin>(smem_u32(&bar_q[1]), nq & 1, abort_flag, p.dev_status);
      if (!ok) break;
      tc_fence_after();
      if (n1 > 0) {
        issue_qk<D, F8>(S_t[1], qd[1], kd[st0], qtd[1], ktd[st0], e);
        mma_commit_elect(smem_u32(&bar_s[1]), e);
      }
      if (!kOneKV) mma_commit_elect(smem_u32(&bar_k_empty[st0]), e);
      if (n1 <= 1) mma_commit_elect(smem_u32(&bar_q_empty[1]), e);
      // Order on the tensor core: PV0(j) S0(j+1) PV1(j) S1(j+1), each warpgroup only for
      // the tiles its rows can see (its fully masked tiles are never computed). First the
      // tiles after which both warpgroups still have one (the straight-line body), then
      // the last one or two, where a warpgroup may stop or sit out.
      const int nb = n0 < n1 ? n0 : n1;
      int j = 0;
      // kWin, d = 64: all by the second loop. What the instruction cache does not hold costs more
      // there than the branches (88 -> 84 us; d = 128: 105 -> 108).
      constexpr bool kStraight = !(kWin && D == 64);
      // kWin: first the second loop for the tiles with hidden keys, then both in turn.
      int until = kWin ? last_hid + 1 : n;
      do {
        if (!kWin || j >= until) {
          for (; kStraight && j + 1 < nb; ++j) {
            const int gj = gt + j;
            const int st = gj % NS;
            const int st1 = (gj + 1) % NS;
            if (!kOneKV && !all_wait<kWin>(smem_u32(&bar_v[st]), (gj / NS) & 1, abort_flag, p.dev_status)) {
              ok = false;
              break;
            }
            if (!pv(0, st, j, g0)) {
              ok = false;
              break;
            }
            if (!all_wait<kWin>(smem_u32(&bar_k[st1]), ((gj + 1) / NS) & 1, abort_flag, p.dev_status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_qk<D, F8>(S_t[0], qd[0], kd[st1], qtd[0], ktd[st1], e);
            mma_commit_elect(smem_u32(&bar_s[0]), e);
            if (j + 2 == n0) mma_commit_elect(smem_u32(&bar_q_empty[0]), e);
            if (!pv(1, st, j, g1)) {
              ok = false;
              break;
            }
            mma_commit_elect(smem_u32(&bar_kv_empty[st]), e);
            issue_qk<D, F8>(S_t[1], qd[1], kd[st1], qtd[1], ktd[st1], e);
            mma_commit_elect(smem_u32(&bar_s[1]), e);
            if (!kOneKV) mma_commit_elect(smem_u32(&bar_k_empty[st1]), e);
            if (j + 2 == n1) mma_commit_elect(smem_u32(&bar_q_empty[1]), e);
          }
          until = n;
        }
        for (; ok && j < until; ++j) {
          const int gj = gt + j;
          const int st = gj % NS;
          const int st1 = (gj + 1) % NS;
          const bool act0 = j < n0, act1 = j < n1;
          const bool more0 = j + 1 < n0, more1 = j + 1 < n1;
          if (!kOneKV && !all_wait<kWin>(smem_u32(&bar_v[st]), (gj / NS) & 1, abort_flag, p.dev_status)) {
            ok = false;
            break;
          }
          if constexpr (kWin) {
            // Rows of V that no row of the sequence sees, and those behind its last key: what they
            // hold must not meet a weight of zero as NaN (V has landed: waited for above, or with K).
            const bool end = j == n - 1 && tail_row < kBlockN;
            if (end || j <= last_hid) {
              const int64_t kv0 = (int64_t)key_tile<true>(w, j) * kBlockN;
              auto row_of = [&](int64_t key) -> int {
                return key <= kv0 ? 0 : key - kv0 < kBlockN ? (int)(key - kv0) : kBlockN;
              };
              const int from = row_of(p.sinks), to = j <= last_hid ? row_of(hid_end) : 0;
              const int behind = end ? tail_row : kBlockN;
              constexpr int kRow = C::kVBoxBytes / kBlockN;  // bytes of a row in one box
              for (int b = 0; b < C::kVBoxes; ++b)
                for (int o = lane * 16; o < kBlockN * kRow; o += 32 * 16) {
                  const int r = o / kRow;
                  if ((r >= from && r < to) || r >= behind)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                     sV(st) + b * C::kVBoxBytes + o),
                                 "r"(0)
                                 : "memory");
                }
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          // warpgroup 0
          if (act0) {
            if (!pv(0, st, j, g0)) {
              ok = false;
              break;
            }
            if (more0) {
              if (!all_wait<kWin>(smem_u32(&bar_k[st1]), ((gj + 1) / NS) & 1, abort_flag,
                             p.dev_status)) {
                ok = false;
                break;
              }
              tc_fence_after();
              issue_qk<D, F8>(S_t[0], qd[0], kd[st1], qtd[0], ktd[st1], e);
              mma_commit_elect(smem_u32(&bar_s[0]), e);
              if (!kOneKV && !more1) mma_commit_elect(smem_u32(&bar_k_empty[st1]), e);
              if (j + 2 == n0) mma_commit_elect(smem_u32(&bar_q_empty[0]), e);
            } else {
              mma_commit_elect(smem_u32(&bar_o[0]), e);
            }
          }
          // warpgroup 1
          if (act1) {
            if (!pv(1, st, j, g1)) {
              ok = false;
              break;
            }
          }
          mma_commit_elect(smem_u32(&bar_kv_empty[st]), e);  // every PV of this tile issued
          if (act1) {
            if (more1) {
              if (!more0 && !all_wait<kWin>(smem_u32(&bar_k[st1]), ((gj + 1) / NS) & 1, abort_flag,
                                       p.dev_status)) {
                ok = false;
                break;
              }
              tc_fence_after();
              issue_qk<D, F8>(S_t[1], qd[1], kd[st1], qtd[1], ktd[st1], e);
              mma_commit_elect(smem_u32(&bar_s[1]), e);
              if (!kOneKV) mma_commit_elect(smem_u32(&bar_k_empty[st1]), e);
              if (j + 2 == n1) mma_commit_elect(smem_u32(&bar_q_empty[1]), e);
            } else {
              mma_commit_elect(smem_u32(&bar_o[1]), e);
            }
          }
        }
      } while (kWin && ok && j < n);
      gt += n;
      g0 += n0;
      g1 += n1;
      ++nq;
    }
    // Drain: every MMA issued by this warp is complete before TMEM is freed.
    mma_commit_elect(smem_u32(&bar_drain), e);
    mbar_wait(smem_u32(&bar_drain), 0, nullptr, p.dev_status);
  }
  } else {
    // ------------------------------------------------------------ softmax / epilogue
    if constexpr (kWin) take_registers<kSoftmaxRegs>();
    const int wg = (warp - 4) >> 2;            // 0 or 1
    const int row = ((warp & 3) << 5) + lane;  // TMEM lane == row within the tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t S_row = tmem + wg * 128 + lane_off;
    const uint32_t O_row = tmem + 256 + wg * 128 + lane_off;
    float4* stage = reinterpret_cast<float4*>(stage_base + (warp - 4) * 4096);
    int ni = 0, nq = 0, gt = 0;
    bool ok = true;
    while (ok) {
      const int slot = ni & 1;
      ok = __all_sync(0xFFFFFFFFu, thread_wait<kWin>(smem_u32(&bar_item_full[slot]), (ni >> 1) & 1,
                                              abort_flag, p.dev_status));
      if (!ok) break;
      const int it = item_slot[slot];
      Item w;
      if constexpr (kWin) w = s_work[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_item_empty[slot]));
      ++ni;
      if (it < 0) break;
      if constexpr (!kWin) {
        bool bad;
        decode_item<kWin>(p, it, w, &bad);
      }
      const int n_tiles = wg == 0 ? w.n0 : w.n1;  // tiles this warpgroup's rows can see
      const int64_t Lq = w.Lq, Lk = w.Lk;
      int64_t first = w.q_lo + wg * kBlockM;  // this warpgroup's first row and its head
      if constexpr (kWin) {
        first = w.q_lo + wg * w.dr;
        w.h += wg * w.dh;
      }
      const int64_t i = first + row;  // query row within the sequence
      int64_t limit = Lk;                            // keys [0, limit) visible to this row
      if (p.causal) {
        const int64_t lim = i + (Lk - Lq) + 1;
        limit = lim < limit ? lim : limit;
      }
      // exp2-domain factor and natural scale of this row's scores; the e4m3 path folds
      // in the row's q scale and the KV head's k scale (S is a product of codes).
      float c = p.scale_log2, sc = p.scale;
      if constexpr (F8) {
        const float f =
            ((i >= 0 && i < Lq) ? p.q_scale[(w.q_start + i) * p.hq + w.h] : 1.f) * p.k_scale[w.g];
        c *= f;
        sc *= f;
      }
      // kWin: keys [win_lo, limit) and [0, sinks) are visible to this row
      int64_t win_lo = 0;
      if constexpr (kWin) win_lo = i + (Lk - Lq) + 1 - p.window;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < n_tiles; ++j) {
        const int gj = gt + j;
        // tcgen05.ld/st are warp-collective: leave the loop as a whole warp.
        ok = __all_sync(0xFFFFFFFFu, thread_wait<kWin>(smem_u32(&bar_s[wg]), gj & 1, abort_flag,
                                                p.dev_status));
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[128];
        float part_max[4];  // TMEM returns each 32-column chunk's max with the data
  #pragma unroll
        for (int q4 = 0; q4 < 4; ++q4)
          part_max[q4] =
              tmem_ld32_max(S_row + q4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[q4 * 32]));
        tmem_ld_wait();
        float* s = reinterpret_cast<float*>(sr);
        const int64_t kv0 = (int64_t)key_tile<kWin>(w, j) * kBlockN;
        float tile_max = fmaxf(fmax3(part_max[0], part_max[1], part_max[2]), part_max[3]);
        if constexpr (kWin) {
          if (__any_sync(0xFFFFFFFFu, kv0 + kBlockN > limit ||
                                          (kv0 < win_lo && kv0 + kBlockN > p.sinks))) {
            // visible columns of the tile: [0, sk) and [lo, lim)
            const int64_t span = limit - kv0, from = win_lo - kv0, kept = p.sinks - kv0;
            const int lim = span < 128 ? (int)(span < 0 ? 0 : span) : 128;
            const int lo = from > 0 ? (int)(from < 128 ? from : 128) : 0;
            const int sk = kept > 0 ? (int)(kept < 128 ? kept : 128) : 0;
            // one bit per column: a test and a select each, where three comparisons took
            // twice as long
            auto below = [](int n, int c0) -> uint32_t {  // columns c0 .. c0 + 31 under n
              const int b = n - c0;
              return b <= 0 ? 0u : b >= 32 ? 0xFFFFFFFFu : (1u << b) - 1u;
            };
            // words that all rows see keep the maximum that came with them
  #pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t see = below(lim, 32 * q) & (~below(lo, 32 * q) | below(sk, 32 * q));
              if (__all_sync(0xFFFFFFFFu, see == 0xFFFFFFFFu)) continue;
  #pragma unroll
              for (int cc = 0; cc < 32; ++cc)
                if (!((see >> cc) & 1u)) s[32 * q + cc] = -INFINITY;
              part_max[q] = row_max<32>(s + 32 * q);
            }
            tile_max = fmaxf(fmax3(part_max[0], part_max[1], part_max[2]), part_max[3]);
          }
        } else if (kv0 + kBlockN > limit) {  // masked columns must not count in the max
          const int64_t lim = limit - kv0;
  #pragma unroll
          for (int cc = 0; cc < 128; ++cc)
            if (cc >= lim) s[cc] = -INFINITY;
          tile_max = row_max<128>(s);
        }
        const float m_new = fmaxf(m_ref, tile_max);
        const bool resc = (m_new - m_ref) * c > 8.0f;  // false for -inf - -inf (NaN)
        float alpha = 1.f;
        if (resc) {
          alpha = ex2_approx((m_ref - m_new) * c);  // 0 when m_ref = -inf
          l *= alpha;
          m_ref = m_new;
        }
        const float neg_mc = (m_ref == -INFINITY) ? 0.f : -m_ref * c;
        auto rescale = [&]() {
          // Rescale O (its previous PV finished: it was issued before this tile's S MMA,
          // whose completion this thread observed).
          if (j > 0 && __any_sync(0xFFFFFFFFu, resc)) {
  #pragma unroll (kWin ? 1 : D / 16)
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t o[16];
              tmem_ld16(O_row + c0, o);
              tmem_ld_wait();
  #pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(O_row + c0, o);
            }
          }
        };
        if constexpr (kWin) {
          // The weights of 64 keys go to TMEM and are announced while the others are computed.
          // Sums in the order of the kernel without a window.
          float2 acc[4] = {};
          float l_a = 0.f;
          exp2_pack_acc<64>(sr, c, neg_mc, acc);
          if constexpr (D >= 128) {
            l_a = sum_of(acc);
  #pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = make_float2(0.f, 0.f);
          }
          tmem_st32(S_row, *reinterpret_cast<const uint32_t(*)[32]>(&sr[0]));
          rescale();
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(smem_u32(&bar_half[wg]));
          exp2_pack_acc<64>(sr + 64, c, neg_mc, acc);
          tmem_st32(S_row + 32, *reinterpret_cast<const uint32_t(*)[32]>(&sr[64]));
          l += D >= 128 ? l_a + sum_of(acc) : sum_of(acc);
        } else {
        // P packed as bf16 pairs in place (over sr[0..63], or sr[0..31] and sr[64..95]).
        if constexpr (D >= 128) {
          // Two halves: the first half of P goes to TMEM while the second is computed
          // (and fewer values stay live, which at d = 128 removes most spills).
          const float l_a = exp2_pack_sum<64>(sr, c, neg_mc);
          tmem_st32(S_row, *reinterpret_cast<const uint32_t(*)[32]>(&sr[0]));
          const float l_b = exp2_pack_sum<64>(sr + 64, c, neg_mc);
          tmem_st32(S_row + 32, *reinterpret_cast<const uint32_t(*)[32]>(&sr[64]));
          l += l_a + l_b;
        } else {
          l += exp2_pack_sum<128>(sr, c, neg_mc);
  #pragma unroll
          for (int q4 = 0; q4 < 2; ++q4)
            tmem_st32(S_row + q4 * 32, *reinterpret_cast<const uint32_t(*)[32]>(&sr[q4 * 32]));
        }
        rescale();
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&bar_p[wg]));
      }
      // ---- epilogue: out = O / l, lse = m * scale + ln l ----
      if (ok && n_tiles > 0)
        ok = __all_sync(0xFFFFFFFFu,
                        thread_wait<kWin>(smem_u32(&bar_o[wg]), nq & 1, abort_flag, p.dev_status));
      if (!ok) break;
      tc_fence_after();
      const float inv_l = (l > 0.f) ? 1.f / l : 0.f;
      if constexpr (kWin) {
        // 128 bytes of each of the warp's 32 rows at a time (64 bf16 or 32 fp32 columns; less in
        // d = 80's tail): one row per thread out of TMEM, through the warp's staging slice,
        // and from there by one TMA store, so that the warp goes on with the next item while the
        // rows are still on their way. Rows that end inside the 32 (a sequence's last) and the tail
        // leave by plain stores. bf16: each value rounded to nearest even, the only rounding.
        const int64_t row0 = first + (warp & 3) * 32;  // this warp's first row
        if (row0 + 32 > 0 && row0 < Lq) {              // uniform: row0 is a multiple of 32
          const bool whole = row0 + 32 <= Lq;
          const uint32_t slice = smem_u32(stage);
          auto columns = [&](auto out_bf16) {
            constexpr bool kHalf = decltype(out_bf16)::value;
            constexpr int kCols = kHalf ? 64 : 32, kSize = kHalf ? 2 : 4;
#pragma unroll (D % 64 == 0 ? 1 : D / kCols + 1)
            for (int c0 = 0; c0 < D; c0 += kCols) {
              const int cw = D - c0 < kCols ? D - c0 : kCols;  // kCols, or 16 for the tail
              uint32_t o[kCols];
#pragma unroll
              for (int h = 0; h < kCols; h += 32) {
                if (h >= cw) continue;
                if (n_tiles > 0) {
                  if (cw - h >= 32)
                    tmem_ld32(O_row + c0 + h, *reinterpret_cast<uint32_t(*)[32]>(&o[h]));
                  else
                    tmem_ld16(O_row + c0 + h, *reinterpret_cast<uint32_t(*)[16]>(&o[h]));
                } else {
#pragma unroll
                  for (int q = 0; q < 32; ++q) o[h + q] = 0u;
                }
              }
              tmem_ld_wait();
              if (lane == 0) bulk_wait_read_all();  // the slice's last store has read it
              __syncwarp();
#pragma unroll
              for (int q = 0; q < 8; ++q)  // 16 bytes; the order is TMA's 128-byte swizzle
                if (q * 16 < cw * kSize) {
                  uint32_t v[4];
#pragma unroll
                  for (int z = 0; z < 4; ++z) {
                    if constexpr (kHalf)
                      v[z] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * z]) * inv_l,
                                         __uint_as_float(o[8 * q + 2 * z + 1]) * inv_l);
                    else
                      v[z] = __float_as_uint(__uint_as_float(o[4 * q + z]) * inv_l);
                  }
                  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                   slice + lane * 128 + ((q ^ (lane & 7)) << 4)),
                               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                               : "memory");
                }
              if (whole && cw == kCols) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                  tma_store_3d(&maps.o, slice, c0, w.h, (int)(w.q_start + row0));
                  bulk_commit();
                }
              } else {
                __syncwarp();
                const int lpr = cw * kSize / 16;  // lanes per row segment
                for (int rr = 0; rr < 32; rr += 32 / lpr) {
                  const int r = rr + lane / lpr, q = lane % lpr;
                  const uint4 v = reinterpret_cast<const uint4*>(stage)[r * 8 + (q ^ (r & 7))];
                  const int64_t ii = row0 + r;
                  if (ii < Lq)
                    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p.out) +
                                              (((w.q_start + ii) * p.hq + w.h) * (int64_t)D + c0) *
                                                  kSize + 16 * q) = v;
                }
                __syncwarp();
              }
            }
          };
          if (p.out_bf16)
            columns(std::true_type());
          else
            columns(std::false_type());
        }
      } else {
      // Rows leave TMEM one per thread; this warp's 4 KB staging slice turns them into
      // whole 128-byte row segments, so each store instruction writes full lines.
      const int64_t row0 = first + (warp & 3) * 32;  // this warp's first row
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        constexpr int kW = 32;
        const int cw = (D - c0 < kW) ? D - c0 : kW;  // 32, or 16 for the d = 80 tail
        uint32_t o[32];
        if (n_tiles > 0) {
          if (cw == 32) {
            tmem_ld32(O_row + c0, o);
          } else {
            tmem_ld16(O_row + c0, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
          }
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) o[q] = 0u;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < cw / 4)
            stage[lane * 8 + (q ^ (lane & 7))] = make_float4(
                __uint_as_float(o[4 * q]) * inv_l, __uint_as_float(o[4 * q + 1]) * inv_l,
                __uint_as_float(o[4 * q + 2]) * inv_l, __uint_as_float(o[4 * q + 3]) * inv_l);
        __syncwarp();
        const int lpr = cw / 4;  // lanes per row segment
        for (int rr = 0; rr < 32; rr += 32 / lpr) {
          const int r = rr + lane / lpr, q = lane % lpr;
          const float4 v = stage[r * 8 + (q ^ (r & 7))];
          const int64_t ii = row0 + r;
          if (ii >= 0 && ii < Lq)
            *reinterpret_cast<float4*>(p.out + ((w.q_start + ii) * p.hq + w.h) * (int64_t)D +
                                       c0 + 4 * q) = v;
        }
        __syncwarp();
      }
      }
      if (i >= 0 && i < Lq && p.lse != nullptr)
        p.lse[(w.q_start + i) * p.hq + w.h] =
            (l > 0.f) ? m_ref * sc + log2f(l) * 0.69314718055994531f : -INFINITY;
      gt += n_tiles;
      if (n_tiles > 0) ++nq;
    }
    if constexpr (kWin) {
      if (lane == 0) bulk_wait_read_all();  // shared memory stays until then
    }
  }

  tc_fence_before();
  __syncthreads();
  if (kWin && tid == 0 && *abort_flag && p.dev_status != nullptr)
    atomicOr(p.dev_status, kDevTimeout);  // a wait ran out
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

__global__ void f32_to_bf16_kernel(const float4* __restrict__ in, uint2* __restrict__ out,
                                   int64_t n4) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n4;
       i += (int64_t)gridDim.x * blockDim.x) {
    const float4 v = in[i];
    out[i] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

template <int D, bool F8 = false, bool kWin = false>
cudaError_t launch_d(const AttnArgs& a, int* drv_err, cudaStream_t stream) {
  using C = AttnCfg<D, F8>;
  MapsFor<kWin> maps;
  // es: bytes per value (2: bf16, 1: e4m3 q / k, 4: fp32 out)
  auto make = [&](CUtensorMap* m, const void* base, int64_t tokens, int heads, uint32_t box0,
                  CUtensorMapSwizzle sw, int es = 2, int box_rows = kBlockN) -> bool {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)heads, (uint64_t)tokens};
    const uint64_t strides[2] = {(uint64_t)D * es, (uint64_t)heads * D * es};
    const uint32_t box[3] = {box0, 1, (uint32_t)box_rows};
    CUresult r = encode_tensor_map(m,
                                   es == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                                   3, const_cast<void*>(base), dims, strides, box, sw);
    if (r != CUDA_SUCCESS) {
      *drv_err = (int)r;
      return false;
    }
    return true;
  };
  const int64_t tq = a.total_q > 0 ? a.total_q : 1, tk = a.total_k > 0 ? a.total_k : 1;
  constexpr int qk_es = F8 ? 1 : 2;
  if (!make(&maps.q, a.q, tq, a.hq, C::kQKCols, CU_TENSOR_MAP_SWIZZLE_128B, qk_es) ||
      !make(&maps.k, a.k, tk, a.hkv, C::kQKCols, CU_TENSOR_MAP_SWIZZLE_128B, qk_es) ||
      !make(&maps.v, a.v, tk, a.hkv, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if constexpr (C::kTail != 0) {
    if (!make(&maps.q_t, a.q, tq, a.hq, 16, CU_TENSOR_MAP_SWIZZLE_32B) ||
        !make(&maps.k_t, a.k, tk, a.hkv, 16, CU_TENSOR_MAP_SWIZZLE_32B) ||
        !make(&maps.v_t, a.v, tk, a.hkv, 32, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  } else {
    maps.q_t = maps.q;
    maps.k_t = maps.k;
    maps.v_t = maps.v;
  }
  if constexpr (kWin) {
    if (!make(&maps.o, a.out, tq, a.hq, a.out_bf16 ? 64 : 32, CU_TENSOR_MAP_SWIZZLE_128B,
              a.out_bf16 ? 2 : 4, 32))
      return cudaErrorInvalidValue;
  }
  ParamsFor<kWin> p;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.out = a.out;
  p.lse = a.lse;
  p.dev_status = a.dev_status;
  p.total_q = a.total_q;
  p.total_k = a.total_k;
  p.batch = a.batch;
  p.max_seqlen_q = a.max_seqlen_q;
  p.max_seqlen_k = a.max_seqlen_k;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.causal = a.causal;
  p.pairs_max = (a.max_seqlen_q + 2 * kBlockM - 1) / (2 * kBlockM);
  p.scale = a.scale;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.q_scale = a.q_scale;
  p.k_scale = a.k_scale;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if constexpr (kWin) {
    p.window = a.window;
    p.sinks = a.sinks;
    p.out_bf16 = a.out_bf16 ? 1 : 0;
    // the bound may be any int; no sequence is longer than all rows
    const int64_t longest = a.max_seqlen_q < a.total_q ? a.max_seqlen_q : a.total_q;
    const int tiles = (int)((longest + kBlockM - 1) / kBlockM);
    p.pairs_max = (tiles + 1) / 2;
    p.pairing = (int64_t)a.batch * tiles * a.hq <= sms ? WindowParams::kSolo
                : (a.hq / a.hkv) % 2 == 0              ? WindowParams::kHeads
                                                       : WindowParams::kRows;
    if (p.pairing != WindowParams::kRows) p.pairs_max = tiles;
  }
  int heads = a.hq;  // items per (sequence, rows)
  if constexpr (kWin) heads = p.pairing == WindowParams::kHeads ? a.hq / 2 : a.hq;
  const int64_t items = (int64_t)a.batch * p.pairs_max * heads;
  if (items == 0) return cudaSuccess;
  if (items > 0x7FFFFFFF || a.work_counter == nullptr) return cudaErrorInvalidConfiguration;
  p.work_counter = a.work_counter;
  p.n_items = (int)items;
  // One persistent CTA per SM (the kernel's shared memory and TMEM allow one).
  const int grid = (int)(items < sms ? items : sms);
  e = cudaFuncSetAttribute(attn_fwd_kernel<D, F8, kWin>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::kSmemBytes);
  if (e != cudaSuccess) return e;
  if constexpr (kWin) {
    static std::atomic<int> known{0};
    int regs = 0;
    e = ask_once(known, &regs, [](int* n) {
      cudaFuncAttributes f;
      const cudaError_t err = cudaFuncGetAttributes(&f, attn_fwd_kernel<D, F8, kWin>);
      if (err == cudaSuccess) *n = f.numRegs;
      return err;
    });
    if (e != cudaSuccess) return e;
    if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  if (kWin && items <= sms) {
    p.work_counter = nullptr;  // one item per CTA: none to hand out, nothing to zero first
  } else {
    e = cudaMemsetAsync(a.work_counter, 0, sizeof(uint32_t), stream);
    if (e != cudaSuccess) return e;
  }
  if constexpr (kWin) {
    if (p.work_counter == nullptr)  // else the kernel follows the counter's memset, not a kernel
      return launch_ahead(attn_fwd_kernel<D, F8, kWin>, dim3(grid), kAttnThreads, C::kSmemBytes,
                          stream, maps, p);
  }
  attn_fwd_kernel<D, F8, kWin><<<grid, kAttnThreads, C::kSmemBytes, stream>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd(const AttnArgs& a, int* drv_err, cudaStream_t stream) {
  if (a.window > 0) {
    if (a.fp8) return cudaErrorInvalidValue;
    switch (a.d) {
      case 64: return launch_d<64, false, true>(a, drv_err, stream);
      case 80: return launch_d<80, false, true>(a, drv_err, stream);
      case 128: return launch_d<128, false, true>(a, drv_err, stream);
      default: return cudaErrorInvalidValue;
    }
  }
  switch (a.d) {
    case 64: return a.fp8 ? cudaErrorInvalidValue : launch_d<64>(a, drv_err, stream);
    case 80: return a.fp8 ? cudaErrorInvalidValue : launch_d<80>(a, drv_err, stream);
    case 128: return a.fp8 ? launch_d<128, true>(a, drv_err, stream)
                           : launch_d<128>(a, drv_err, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_f32_to_bf16(const float* in, void* out, int64_t n, cudaStream_t stream) {
  // n is a multiple of 4 (head_dim is), pointers 16 / 8-byte aligned.
  const int64_t n4 = n / 4;
  if (n4 == 0) return cudaSuccess;
  int blocks = (int)((n4 + 255) / 256);
  if (blocks > 152 * 16) blocks = 152 * 16;
  f32_to_bf16_kernel<<<blocks, 256, 0, stream>>>(reinterpret_cast<const float4*>(in),
                                                  reinterpret_cast<uint2*>(out), n4);
  return cudaGetLastError();
}

}  // namespace tts
