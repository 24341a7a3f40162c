// q4_attn.cu — decode attention over a paged cache held in 4 bits.
//
// A CTA takes a query row; its warps take keys in turn, a lane D / 32 values of each, with a
// running maximum and sum; the warps' states are added up at the end.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/decode_attn.h"
#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace {

constexpr int kWarps = 4;

struct Q4Params {
  const float* q;
  const uint8_t* pool;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* q_pos;
  float* out;
  float* lse;
  int32_t* dev_status;
  int B, T, Hq, Hkv, group, log2_bs, max_blocks, num_blocks, window, causal;
  float qscale, softcap2;
  long long page_bytes;
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps) q4_kernel(const Q4Params p) {
  constexpr int V = D / 32;  // values of a lane: V / 2 bytes side by side
  __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
  const int h = blockIdx.x % p.Hq, bt = blockIdx.x / p.Hq, t = bt % p.T, b = bt / p.T;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int kv = h / (p.Hq / p.Hkv), bs = 1 << p.log2_bs, ng = D / p.group;
  const long long cap = (long long)p.max_blocks << p.log2_bs;
  int flag = 0;
  long long L = p.seq_lens[b];
  if (L < 0 || L > cap) {
    flag |= DA_DEV_BAD_SEQ_LEN;
    L = L < 0 ? 0 : cap;
  }
  long long qp = L - p.T;
  bool empty = false;
  if (p.q_pos) {
    qp = p.q_pos[b];
    if (qp < 0) flag |= DA_DEV_BAD_QPOS, empty = true;
  }
  qp += t;
  long long lo = p.window > 0 && qp >= p.window ? qp - p.window + 1 : 0;
  long long hi = p.causal && qp + 1 < L ? qp + 1 : L;
  if (empty) hi = lo;
  const long long row = ((long long)b * p.T + t) * p.Hq + h;
  float q[V];
  for (int i = 0; i < V; ++i) q[i] = p.q[row * D + lane * V + i] * p.qscale;
  float m = -INFINITY, l = 0.f, o[V] = {};
  for (long long key = lo + warp; key < hi; key += kWarps) {
    const int blk = p.table[(long long)b * p.max_blocks + (key >> p.log2_bs)];
    if (blk < 0 || blk >= p.num_blocks) {
      flag |= DA_DEV_BAD_BLOCK;
      continue;
    }
    const int r = (int)(key & (bs - 1));
    const uint8_t* page = p.pool + ((long long)blk * p.Hkv + kv) * p.page_bytes;
    const int d = lane * V, byte = d / 2;
    const uint8_t* at = page + r * (D / 2) + ((byte / 16) ^ da::piece_xor<D>(r)) * 16 + byte % 16;
    const __half2* par = reinterpret_cast<const __half2*>(page + bs * D) + r * ng + d / p.group;
    const float2 kp = __half22float2(par[0]), vp = __half22float2(par[bs * ng]);
    float s = 0.f;
    for (int i = 0; i < V; ++i)
      s += q[i] * fmaf((float)(at[i / 2] >> (4 * (i % 2)) & 15), kp.x, kp.y);
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (p.softcap2 > 0.f) s = p.softcap2 * tanhf(s / p.softcap2);
    // a NaN score leaves the maximum alone and makes the sums NaN
    const float m2 = fmaxf(m, s), c = m == -INFINITY ? 0.f : exp2f(m - m2);
    const float w = s == -INFINITY ? 0.f : exp2f(s - m2);
    m = m2;
    l = l * c + w;
    for (int i = 0; i < V; ++i)
      o[i] = o[i] * c + w * fmaf((float)(at[bs * (D / 2) + i / 2] >> (4 * (i % 2)) & 15), vp.x, vp.y);
  }
  for (int i = 0; i < V; ++i) so[warp][lane * V + i] = o[i];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  if (flag && lane == 0 && p.dev_status) atomicOr(p.dev_status, flag);
  __syncthreads();
  float M = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  auto share = [&](int w) { return sm[w] == M ? 1.f : sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - M); };
  for (int w = 0; w < kWarps; ++w) total += sl[w] * share(w);
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += so[w][d] * share(w);
    p.out[row * D + d] = total == 0.f ? 0.f : x / total;
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[row] = total == 0.f ? -INFINITY : (M + log2f(total)) * 0.6931471805599453f;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check(const da_params* p, int group, int q_len) {
  int st = da::check_paged(p);
  if (st == DA_OK) st = da::check_q4(p, group);
  if (st != DA_OK) return st;
  if (q_len < 1) return DA_ERR_INVALID;
  if ((long long)q_len * p->num_q_heads * 1024 > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

}  // namespace

extern "C" {

size_t decode_attn_paged_q4_workspace_size(const da_params* p, int32_t q_len) {
  return check(p, da::kQ4MinGroup, q_len) == DA_OK ? 256 : 0;
}

int decode_attn_paged_q4(const da_params* p, int32_t group, int32_t q_len, const float* q,
                         const uint8_t* pool, const int32_t* block_table,
                         const int32_t* seq_lens, const int32_t* q_pos, float* out, float* lse,
                         void* workspace, size_t workspace_bytes, int32_t* dev_status,
                         void* stream) {
  const int st = check(p, group, q_len);
  if (st != DA_OK) return st;
  if (!q || !pool || !block_table || !seq_lens || !out) return DA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || (q_pos && !aligned(q_pos, 4)) || (lse && !aligned(lse, 4)) ||
      (dev_status && !aligned(dev_status, 4)) || !aligned(workspace, 256))
    return DA_ERR_INVALID;
  if (!workspace && workspace_bytes) return DA_ERR_INVALID;
  const long long values = (long long)p->batch * q_len * p->num_q_heads * p->head_dim;
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
  if ((qa < oa ? oa - qa : qa - oa) < (unsigned long long)values * 4) return DA_ERR_INVALID;
  if (workspace && workspace_bytes < decode_attn_paged_q4_workspace_size(p, q_len))
    return DA_ERR_WORKSPACE;
  if (p->batch == 0) return DA_OK;
  Q4Params k = {};
  k.q = q;
  k.pool = pool;
  k.table = block_table;
  k.seq_lens = seq_lens;
  k.q_pos = q_pos;
  k.out = out;
  k.lse = lse;
  k.dev_status = dev_status;
  k.B = p->batch;
  k.T = q_len;
  k.Hq = p->num_q_heads;
  k.Hkv = p->num_kv_heads;
  k.group = group;
  while ((1 << k.log2_bs) < p->block_size) ++k.log2_bs;
  k.max_blocks = p->max_blocks_per_seq;
  k.num_blocks = p->num_blocks;
  k.window = p->sliding_window;
  k.causal = p->causal;
  k.qscale = da::base2_scale(p);
  k.softcap2 = p->softcap * 1.4426950408889634f;
  k.page_bytes = da::q4_page_bytes(p->block_size, p->head_dim, group);
  const unsigned grid = (unsigned)p->batch * q_len * p->num_q_heads;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->head_dim == 64) q4_kernel<64><<<grid, 32 * kWarps, 0, s>>>(k);
  else if (p->head_dim == 128) q4_kernel<128><<<grid, 32 * kWarps, 0, s>>>(k);
  else q4_kernel<256><<<grid, 32 * kWarps, 0, s>>>(k);
  return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

}  // extern "C"
