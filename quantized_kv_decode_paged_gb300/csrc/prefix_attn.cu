// prefix_attn.cu — decode attention of a batch that shares the pages of a
// long prefix.
//
// Row (b, t, h) attends to the keys [lo, hi) its masks leave: softmax over
// s_j = scale <q, k_j> (softcap on top), out = sum p_j v_j / sum p_j and
// lse = m + ln sum e^(s_j - m), kept as the running state (m, l, o) of one
// pass over the keys in base-2 units.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/decode_attn.h"
#include "launch.h"
#include "ptx.cuh"

namespace da {

namespace {

constexpr float kInf = INFINITY;
constexpr float kLn2 = 0.6931471805599453f;

// tanh by its identity in 2^x; below 1/2, where the identity's rounding next
// to 1 would cost relative accuracy, by the Taylor series through y^13
// (coefficients 2^2n (2^2n - 1) B_2n / (2n)!): a score keeps f32's relative
// accuracy whatever the cap.
__device__ __forceinline__ float capped(float x, float cap2, float inv_cap2) {
  const float y = x * inv_cap2;
  const float y2 = y * y;
  float t = 21844.f / 6081075.f;
  t = fmaf(t, y2, -1382.f / 155925.f);
  t = fmaf(t, y2, 62.f / 2835.f);
  t = fmaf(t, y2, -17.f / 315.f);
  t = fmaf(t, y2, 2.f / 15.f);
  t = fmaf(t, y2, -1.f / 3.f);
  t = fmaf(t * y2, y, y);
  const float big = 1.f - __fdividef(2.f, ex2_ftz(y * 2.8853900817779268f) + 1.f);
  return cap2 * (fabsf(y) <= 0.5f ? t : big);
}

// Keys [lo, hi) that query token t of sequence b sees; returns device-status
// bits.  The token sits at q_pos[b] + t, by default seq_len - T + t.
__device__ __forceinline__ int row_range(const PrefixParams& p, int b, int t, int& lo, int& hi) {
  int flags = 0;
  const long long cap = (long long)p.max_blocks * p.bs;
  long long L = p.seq_lens[b];
  if (L < 0 || L > cap) {
    flags |= DEV_BAD_SEQ_LEN;
    L = L < 0 ? 0 : cap;
  }
  long long qp = L - p.T + t;
  bool empty = false;
  if (p.q_pos) {
    const int q0 = p.q_pos[b];
    if (q0 < 0) {
      flags |= DEV_BAD_QPOS;
      empty = true;
    }
    qp = (long long)q0 + t;
  }
  const long long l = (p.window > 0 && qp >= p.window) ? qp - p.window + 1 : 0;
  long long h = p.causal ? qp + 1 : L;
  h = h < L ? h : L;
  if (empty || h <= l) {
    lo = hi = 0;
  } else {
    lo = (int)l;
    hi = (int)h;
  }
  return flags;
}

// Page of key k of sequence b (not checked against num_blocks).
__device__ __forceinline__ int page_of(const PrefixParams& p, int b, int k) {
  const int c = k >> p.log2_bs;
  return c < p.prefix_pages ? p.prefix_table[c]
                            : p.block_table[(long long)b * p.max_blocks + c];
}

// One warp's state of a row over keys [k0, k1): lane i holds the values
// [i * D/32, (i + 1) * D/32) of q and o.  Returns device-status bits.
template <int D>
__device__ int attend_row(const PrefixParams& p, int b, int kv, const float (&q)[D / 32], int k0,
                          int k1, float& m, float& l, float (&o)[D / 32]) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  m = -kInf;
  l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  int flags = 0;
  for (int k = k0; k < k1; ++k) {
    const int blk = page_of(p, b, k);
    if (blk < 0 || blk >= p.num_blocks) {
      flags |= DEV_BAD_BLOCK;
      continue;
    }
    const long long at =
        ((((long long)blk << p.log2_bs) + (k & (p.bs - 1))) * p.Hkv + kv) * D + lane * V;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(p.k_pool + at + i));
      s = fmaf(q[i], x.x, fmaf(q[i + 1], x.y, s));
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.qscale;
    if (p.softcap2 > 0.f) s = capped(s, p.softcap2, p.softcap_inv);
    const float mn = fmaxf(m, s);
    const float base = mn == -kInf ? 0.f : mn;
    const float f = exp2f(m - base), w = exp2f(s - base);
    l = fmaf(l, f, w);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(p.v_pool + at + i));
      o[i] = fmaf(o[i], f, w * x.x);
      o[i + 1] = fmaf(o[i + 1], f, w * x.y);
    }
    m = mn;
  }
  return flags;
}

constexpr int kRowWarps = 4;

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) prefix_rows_kernel(const PrefixParams p) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (row >= (long long)p.B * p.T * p.Hq) return;
  const int h = (int)(row % p.Hq);
  const int b = (int)(row / p.Hq / p.T), t = (int)(row / p.Hq % p.T);
  float q[V], o[V], m, l;
#pragma unroll
  for (int i = 0; i < V; ++i) q[i] = p.q[row * D + lane * V + i];
  int lo, hi;
  int flags = row_range(p, b, t, lo, hi);
  flags |= attend_row<D>(p, b, h / p.G, q, lo, hi, m, l, o);
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int i = 0; i < V; ++i) p.out[row * D + lane * V + i] = o[i] * inv;
  if (lane == 0 && p.lse) p.lse[row] = l == 0.f ? -kInf : m * kLn2 + logf(l);
  if (lane == 0 && flags && p.dev_status) atomicOr(p.dev_status, flags);
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.T * p.Hq;
  const long long blocks = (rows + kRowWarps - 1) / kRowWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int grid = (int)blocks;
  if (p.D == 64)
    prefix_rows_kernel<64><<<grid, kRowWarps * 32, 0, stream>>>(p);
  else if (p.D == 128)
    prefix_rows_kernel<128><<<grid, kRowWarps * 32, 0, stream>>>(p);
  else
    prefix_rows_kernel<256><<<grid, kRowWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace da
