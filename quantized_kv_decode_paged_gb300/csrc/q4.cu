// q4.cu — the cache in 4 bits as rows again: cached tokens to f32, f16 or bf16.
//
// A value is scale * code + zero (q4.cuh), one fused multiply-add: in f16 for f16 rows, in f32 and rounded to bf16
// for those.  f16 rows saturate at 65504, which a code's rounding may pass by half a step.
// A thread takes eight codes, one word, so that a warp's loads and its 16- or 32-byte stores
// cover whole sectors; a CTA looks its tokens' pages up once.  HBM bounds long calls.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/decode_attn.h"
#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 128;  // of a CTA
// Words of eight codes of keys and values that a thread has in work at once.
constexpr int kAtOnce = 4;

struct GatherArgs {
  const int32_t* positions;
  const int32_t* token_seq;
  const int32_t* block_table;
  const uint8_t* pool;
  void* k_out;
  void* v_out;
  int N, tokens, Hkv, group;
  uint64_t inv_heads;  // ceil(2^32 / Hkv): r / Hkv = r * inv_heads >> 32, r < 2^16
  int batch, log2_bs, max_blocks, num_blocks;
  long long page_bytes;
  int32_t* dev_status;
};

// Eight values of a word of codes and its param {scale, zero}, stored.
template <typename T>
__device__ __forceinline__ void store_values(T* p, uint32_t codes, uint32_t param) {
  if constexpr (std::is_same<T, __half>::value) {
    // In pairs of f16: 1024 + code less 1024, times the scale, plus the zero, with one rounding; then to f16's range
    // (a NaN stays).  (Through f32, 40,003 tokens x 8 heads x 128 took 58 us, bound by the instructions.)
    uint32_t s2, z2, v[4];
    asm("prmt.b32 %0, %1, %1, 0x1010;" : "=r"(s2) : "r"(param));
    asm("prmt.b32 %0, %1, %1, 0x3232;" : "=r"(z2) : "r"(param));
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // codes i and i + 4
      asm("{\n\t.reg .b32 c;\n\tadd.rn.f16x2 c, %1, %2;\n\tfma.rn.f16x2 %0, c, %3, %4;\n\t"
          "min.NaN.f16x2 %0, %0, %5;\n\tmax.NaN.f16x2 %0, %0, %6;\n\t}"
          : "=r"(v[i])
          : "r"((codes >> (4 * i) & 0x000f000fu) | 0x64006400u), "r"(0xe400e400u), "r"(s2), "r"(z2),
            "r"(0x7bff7bffu), "r"(0xfbfffbffu));
    }
    uint4 w;
    w.x = __byte_perm(v[0], v[1], 0x5410), w.y = __byte_perm(v[2], v[3], 0x5410);
    w.z = __byte_perm(v[0], v[1], 0x7632), w.w = __byte_perm(v[2], v[3], 0x7632);
    *reinterpret_cast<uint4*>(p) = w;
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&param));
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)  // a code is the last bits of 2^23 + code
      x[j] = fmaf(__uint_as_float((codes >> (4 * j) & 15u) | 0x4b000000u) - 8388608.f, f.x, f.y);
    if constexpr (std::is_same<T, float>::value) {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherArgs a) {
  struct Place {
    const uint8_t* page;  // of kv head 0
    int row;              // of the page; -1: none
  };
  __shared__ Place place[kTokens];
  const int n0 = blockIdx.x * a.tokens, tokens = min(a.tokens, a.N - n0);
  da::let_next_grid_start();
  da::wait_for_grid_before();
  if ((int)threadIdx.x < tokens) {
    const int n = n0 + threadIdx.x, seq = a.token_seq ? a.token_seq[n] : n;
    Place x = {a.pool, -1};
    int flag = 0;
    if (seq >= a.batch) {
      flag = DA_DEV_BAD_SEQ;
    } else if (seq >= 0) {
      const int pos = a.positions[n];
      if (pos < 0 || (pos >> a.log2_bs) >= a.max_blocks) {
        flag = DA_DEV_BAD_SEQ_LEN;
      } else {
        const int blk = a.block_table[(long long)seq * a.max_blocks + (pos >> a.log2_bs)];
        if (blk < 0 || blk >= a.num_blocks)
          flag = DA_DEV_BAD_BLOCK;
        else
          x = {a.pool + (long long)blk * a.Hkv * a.page_bytes, pos & ((1 << a.log2_bs) - 1)};
      }
    }
    place[threadIdx.x] = x;
    if (flag && a.dev_status) atomicOr(a.dev_status, flag);
  }
  __syncthreads();
  constexpr int C = D / 8;  // words of a row
  const int bs = 1 << a.log2_bs, ng = D / a.group, items = tokens * a.Hkv * C;
  const int log2_group = 31 - __clz(a.group);
  for (int i0 = threadIdx.x; i0 < items; i0 += kAtOnce * kThreads) {
    uint32_t kc[kAtOnce], vc[kAtOnce], kw[kAtOnce], vw[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kThreads, c = i % C, r = i / C;
      const int t = (int)(((uint64_t)r * a.inv_heads) >> 32), h = r - t * a.Hkv;
      kc[u] = vc[u] = kw[u] = vw[u] = 0;  // codes, scales and zeros of nothing: zeros
      if (i >= items) continue;
      const Place x = place[t];
      if (x.row >= 0) {
        const uint8_t* page = x.page + (long long)h * a.page_bytes;
        const uint8_t* at =
            page + (x.row * (D / 2) + 16 * ((c / 4) ^ da::piece_xor<D>(x.row)) + c % 4 * 4);
        kc[u] = __ldg(reinterpret_cast<const uint32_t*>(at));
        vc[u] = __ldg(reinterpret_cast<const uint32_t*>(at + bs * (D / 2)));
        const uint32_t* par = reinterpret_cast<const uint32_t*>(
            page + (bs * D + (x.row * ng + (c * 8 >> log2_group)) * 4));
        kw[u] = __ldg(par);
        vw[u] = __ldg(par + bs * ng);
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= items) break;
      const long long to = (long long)n0 * a.Hkv * D + (long long)i * 8;
      store_values(static_cast<T*>(a.k_out) + to, kc[u], kw[u]);
      store_values(static_cast<T*>(a.v_out) + to, vc[u], vw[u]);
    }
  }
}

template <typename T>
cudaError_t launch_gather(const GatherArgs& a, int D, cudaStream_t s) {
  const int grid = (a.N - 1) / a.tokens + 1;
  return da::launch_early(D == 64    ? gather_kernel<T, 64>
                          : D == 128 ? gather_kernel<T, 128>
                                     : gather_kernel<T, 256>,
                          grid, kThreads, 0, s, a);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

namespace da {

int check_q4(const da_params* p, int group) {
  if (!p || group <= 0) return DA_ERR_INVALID;
  const int bs = p->block_size, D = p->head_dim;
  if (bs <= 0 || D <= 0) return DA_ERR_INVALID;
  if (bs < 8 || bs > 256 || (bs & (bs - 1)) != 0) return DA_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return DA_ERR_UNSUPPORTED;
  return q4_group_ok(group, D) ? DA_OK : DA_ERR_UNSUPPORTED;
}

}  // namespace da

extern "C" {

size_t decode_attn_q4_page_bytes(int32_t block_size, int32_t head_dim, int32_t group) {
  da_params p = {};
  p.block_size = block_size;
  p.head_dim = head_dim;
  if (da::check_q4(&p, group) != DA_OK) return 0;
  return (size_t)da::q4_page_bytes(block_size, head_dim, group);
}

int decode_attn_gather_paged_q4(const da_params* p, int32_t group, int32_t num_tokens, int32_t type,
                                const int32_t* positions, const int32_t* token_seq,
                                const int32_t* block_table, const uint8_t* pool, void* k_out,
                                void* v_out, int32_t* dev_status, void* stream) {
  int st = da::check_append_params(p);
  if (st == DA_OK) st = da::check_q4(p, group);
  if (st != DA_OK) return st;
  if (type != DA_TYPE_F32 && type != DA_TYPE_F16 && type != DA_TYPE_BF16) return DA_ERR_INVALID;
  if (num_tokens < 0 || (!token_seq && num_tokens != p->batch)) return DA_ERR_INVALID;
  if (!positions || !block_table || !pool || !k_out || !v_out) return DA_ERR_INVALID;
  if (!aligned(pool, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(positions, 4) ||
      !aligned(block_table, 4) || (token_seq && !aligned(token_seq, 4)) ||
      (dev_status && !aligned(dev_status, 4)))
    return DA_ERR_INVALID;
  if (p->num_kv_heads > 4096) return DA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return DA_OK;
  int sms = 0;
  st = da::device_sms(&sms);
  if (st != DA_OK) return st;
  GatherArgs a = {};
  a.positions = positions;
  a.token_seq = token_seq;
  a.block_table = block_table;
  a.pool = pool;
  a.k_out = k_out;
  a.v_out = v_out;
  a.N = num_tokens;
  // Tokens of a CTA: so many that one wave of CTAs, four a processor, has them all where kTokens allow that (a
  // CTA looks its tokens up first, 2 us that others do not hide), and rows of a CTA below 2^16.
  a.tokens = (num_tokens - 1) / (sms * 4) + 1;
  if (a.tokens > kTokens) a.tokens = kTokens;
  if (a.tokens > 65535 / p->num_kv_heads) a.tokens = 65535 / p->num_kv_heads;
  a.Hkv = p->num_kv_heads;
  a.inv_heads = (0x100000000ULL + a.Hkv - 1) / a.Hkv;
  a.group = group;
  a.batch = p->batch;
  while ((1 << a.log2_bs) < p->block_size) ++a.log2_bs;
  a.max_blocks = p->max_blocks_per_seq;
  a.num_blocks = p->num_blocks;
  a.page_bytes = da::q4_page_bytes(p->block_size, p->head_dim, group);
  a.dev_status = dev_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = type == DA_TYPE_F32   ? launch_gather<float>(a, p->head_dim, s)
                          : type == DA_TYPE_F16 ? launch_gather<__half>(a, p->head_dim, s)
                                                : launch_gather<__nv_bfloat16>(a, p->head_dim, s);
  return err == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

}  // extern "C"
