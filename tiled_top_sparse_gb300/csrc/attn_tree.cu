// Attention of a drafted tree of new tokens over the paged grouped-query cache.
//
// Request r's n new tokens are its last n cached rows. Token i sees the new tokens whose bits its
// mask has, and the cached ones before them (with a window: those of its position's window and the
// first ones); its position is past the cached tokens by the number of new tokens that it
// sees besides one (itself).
//
// A block per (token, q head): 128 keys at a time, a key per thread for the scores, a value column
// per thread for the sums.
#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tts {
namespace {

template <bool F8, int D>
__global__ void __launch_bounds__(128) attn_tree_simple_kernel(const AttnDecodeArgs a) {
  wait_for_prior_grids();
  __shared__ float s_q[D], s_p[128], s_red[4];
  __shared__ int s_row[128], s_b, s_n, s_q0;
  const int tid = threadIdx.x, t = blockIdx.x, h = blockIdx.y, g = h / (a.hq / a.hkv);
  if (tid == 0) s_b = -1;
  __syncthreads();
  for (int b = tid; b < a.batch; b += 128) {
    const int q0 = a.cu_q ? a.cu_q[b] : b, q1 = a.cu_q ? a.cu_q[b + 1] : b + 1;
    if (q0 < 0 || q1 < q0 || q1 > a.total_q || q1 - q0 > a.max_q) {
      if (t == 0 && h == 0 && a.dev_status) atomicOr(a.dev_status, kDevBadArg);
    } else if (t >= q0 && t < q1) {
      s_b = b;
      s_n = q1 - q0;
      s_q0 = q0;
    }
  }
  __syncthreads();
  if (s_b < 0) return;
  const int b = s_b, n = s_n;
  int L = a.kv_lens[b];
  if (L < 0 || L > a.max_pages * a.page_size) {
    if (tid == 0 && a.dev_status) atomicOr(a.dev_status, kDevIndexRange);
    L = 0;
  }
  const int base = L - n;
  uint64_t mask = a.tree_mask[t];
  if (n < 64) mask &= (1ull << n) - 1;
  const int pos = base + max(__popcll(mask) - 1, 0);
  for (int i = tid; i < D; i += 128)
    s_q[i] = __uint_as_float((uint32_t) static_cast<const uint16_t*>(
                                 a.q)[((int64_t)t * a.hq + h) * D + i]
                             << 16);
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int k0 = 0; k0 < L; k0 += 128) {
    __syncthreads();
    const int key = k0 + tid;
    const bool see =
        key < L && (key < base ? a.window == 0 || key > pos - a.window || key < a.sinks
                               : ((mask >> (key - base)) & 1) != 0);
    float x = -INFINITY;
    int page = -1;
    if (see) {
      page = a.page_tables[(int64_t)b * a.max_pages + key / a.page_size];
      if (page < 0 || page >= a.num_pages) {
        page = -1;
        if (a.dev_status) atomicOr(a.dev_status, kDevIndexRange);
      }
    }
    if (F8 && page >= 0) {
      const float ks = a.k_scale[(int64_t)page * a.hkv + g], vs = a.v_scale[(int64_t)page * a.hkv + g];
      if (!(ks > 0.f && ks < INFINITY && vs >= 0x1p-80f && vs < INFINITY)) {
        page = -1;
        if (a.dev_status) atomicOr(a.dev_status, kDevBadArg);
      }
    }
    if (page >= 0) {
      const int64_t row = ((int64_t)page * a.hkv + g) * a.page_size + key % a.page_size;
      x = 0.f;
      for (int i = 0; i < D; ++i) {
        float k;
        if constexpr (F8)
          k = float(reinterpret_cast<const __nv_fp8_e4m3*>(a.k_cache)[row * D + i]);
        else
          k = __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.k_cache)[row * D + i] << 16);
        x = fmaf(s_q[i], k, x);
      }
      if constexpr (F8) x *= a.k_scale[(int64_t)page * a.hkv + g];
      x *= a.scale;
    }
    s_row[tid] = page;
    float top = x;
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    if ((tid & 31) == 0) s_red[tid >> 5] = top;
    __syncthreads();
    const float nm = fmaxf(fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])), m);
    const float al = m == -INFINITY ? 0.f : expf(m - nm);
    m = nm;
    s_p[tid] = x == -INFINITY ? 0.f : expf(x - m);
    __syncthreads();
    l *= al;
    o *= al;
    for (int j = 0; j < 128; ++j) {
      const float p = s_p[j];
      l += p;
      if (tid < D && s_row[j] >= 0) {
        const int64_t head = (int64_t)s_row[j] * a.hkv + g;
        const int64_t at = (head * a.page_size + (k0 + j) % a.page_size) * D + tid;
        if constexpr (F8)
          o = fmaf(p * a.v_scale[head], float(reinterpret_cast<const __nv_fp8_e4m3*>(a.v_cache)[at]), o);
        else
          o = fmaf(p, __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.v_cache)[at] << 16), o);
      }
    }
  }
  const int64_t at = (int64_t)t * a.hq + h;
  if (tid < D) {
    const float v = l > 0.f ? o / l : 0.f;
    if (a.out_bf16)
      static_cast<uint16_t*>(a.out)[at * D + tid] = (uint16_t)pack_bf16x2(v, 0.f);
    else
      static_cast<float*>(a.out)[at * D + tid] = v;
  }
  if (tid == 0 && a.lse != nullptr) a.lse[at] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attn_tree_workspace_bytes(int, int, int, int, int) { return 16; }

cudaError_t launch_attn_tree(const AttnDecodeArgs& a, int*, cudaStream_t stream) {
  const dim3 grid((unsigned)a.total_q, (unsigned)a.hq);
  if (a.d == 64)
    return launch_ahead(a.f8 ? attn_tree_simple_kernel<true, 64> : attn_tree_simple_kernel<false, 64>,
                        grid, 128, 0, stream, a);
  return launch_ahead(a.f8 ? attn_tree_simple_kernel<true, 128> : attn_tree_simple_kernel<false, 128>,
                      grid, 128, 0, stream, a);
}

}  // namespace tts
