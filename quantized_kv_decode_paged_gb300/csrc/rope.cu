// rope.cu — what a step does to its new rows before the attention: RMS norm
// of every query and key head, position rotation, and the append of rotated
// keys and plain values to the paged cache, in f16 or in 4 bits.
//
// Mathematics.  A head's row x has D values.  Norm: y_d = x_d r w_d with
// r = 1/sqrt(mean(x^2) + eps).  Rotation of a pair by the angle a:
// (y0 cos a - y1 sin a, y0 sin a + y1 cos a).  a = pos * f turns with f in
// 64-bit fixed point: the low 64 bits of the integer product are the angle
// modulo one turn, exact up to f's own 2^-56 turns a position (a double's).  Its distance from
// the nearest quarter turn is rounded to f32, 2^-24 of a number of at most an eighth, and goes to
// sincospif; the quarter turns swap and negate what comes back.  (The whole angle rounded to
// f32 is off by 2^-25 of half a turn, 9.4e-8, which the small one of sine and cosine shows.)
//
// A CTA takes up to max_tokens tokens: their rd/2 cosines and sines are computed once
// into shared memory and serve all the tokens' heads.  D/16 threads take a row, each
// two 8-value chunks that hold both halves of its 8 pairs: (8c, rd/2 + 8c) or, interleaved,
// (16c, 16c + 8); the chunks past the rotated part pair up without rotation.
// So no value crosses threads but the norm's sum of squares.  A thread's next row is
// loaded before its last one is worked on.  HBM bounds long calls, the host short ones.
//
// Measured (GB300): 16,381 tokens x (32 + 8) heads x 128 from bf16, 470 MB in 74 us, 6.3 TB/s (77.5 to
// 78.3 us a call in a loop); an append of 12,287 tokens x 8 heads x 128 of keys and values, 101 MB in
// 17.8 us a call over the same inputs, 21.6 over changing ones; 128 tokens x 72 heads 4.7 us a call in
// a graph.  In 4 bits those 12,287 tokens take 31 us with cold caches, bound by the instructions (extents of
// the groups, codes): 64 MB.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/decode_attn.h"
#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace {

// What a launch does with its rows: norm and rotation alone, or an append to f16 pages or to
// pages in 4 bits.
enum { kNormRope = 0, kAppend = 1, kAppendQ4 = 2 };

constexpr int kRopeThreads = 256;
// Resident CTAs of an SM (64 registers a thread; 3 and 5, the latter spilling,
// measured 83 and 93-98 us against 79 on 16,381 tokens x 40 heads x 128).
constexpr int kRopeCtas = 4;
constexpr int kMaxTokens = 12;  // of a CTA
// In 4 bits a row takes twice as long, and a CTA's first loads (positions, pages) are better shared by many: those
// 12,287 tokens 44 us with 28, 45 with 20 or 14, 48 with 12.
constexpr int max_tokens(int mode) { return mode == kAppendQ4 ? 28 : kMaxTokens; }
// In 4 bits more registers are live: 12,287 tokens x 8 heads x 128 with their read-back 40 us with three CTAs, 47
// with four (which spill) and 44 with two.
constexpr int rope_ctas(int mode) { return mode == kAppendQ4 ? 3 : kRopeCtas; }

struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;  // element strides of tokens and heads
  const float* qw;
  const float* kw;
  const uint64_t* freqs;
  const int32_t* positions;
  int N, tokens;            // tokens; tokens of a CTA
  int heads;                // rows of a token: q, k and (append) v heads
  uint64_t inv_heads;       // ceil(2^32 / heads): r / heads = r * inv_heads >> 32, r < 2^20
  int Hq, Hk, Hkv, rd, norm;  // Hq, Hk: 0 where q or k is not given
  float eps, woff;
  float* q_out;
  bool wide_out;    // q_out lies on a 32-byte boundary
  uint16_t* k_out;  // norm_rope: [N, Hkv, D]
  // append
  const int32_t* token_seq;
  const int32_t* block_table;
  uint16_t* k_pool;
  uint16_t* v_pool;
  int batch, bs, max_blocks, num_blocks;
  int32_t* dev_status;
  // append in 4 bits
  uint8_t* q4_pool;
  int log2_bs, log2_group;
  long long page_bytes;
};

// Eight values of type T as they lie in memory.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8], const __half*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8], const __nv_bfloat16*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <typename T>
__device__ __forceinline__ Raw<T> load8(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void values8(const Raw<T>& r, float (&x)[8]) {
  if constexpr (std::is_same<T, float>::value) {
    x[0] = __uint_as_float(r.w[0].x), x[1] = __uint_as_float(r.w[0].y);
    x[2] = __uint_as_float(r.w[0].z), x[3] = __uint_as_float(r.w[0].w);
    x[4] = __uint_as_float(r.w[1].x), x[5] = __uint_as_float(r.w[1].y);
    x[6] = __uint_as_float(r.w[1].z), x[7] = __uint_as_float(r.w[1].w);
  } else {
    unpack8(r.w[0], x, static_cast<const T*>(nullptr));
  }
}

// Eight f32 values: in one 32-byte store where the address allows it (two
// 16-byte stores of neighbouring lanes each leave half of every 32-byte sector: 100 us
// against 92 for the 470 MB of 16,381 tokens x 40 heads x 128).
__device__ __forceinline__ void store8(float* p, const float (&x)[8], bool wide) {
  if (wide) {
    da::store_f32x8(p, x);
    return;
  }
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Row n's place in the cache, in rows of the pool; negative: not written
// (padding, or a flag is set).
__device__ __forceinline__ long long cache_row(const RopeArgs& a, int n, int& flag, bool& pad) {
  const int seq = a.token_seq ? a.token_seq[n] : n;
  pad = seq < 0;
  flag = 0;
  if (pad) return -1;
  if (seq >= a.batch) {
    flag = DA_DEV_BAD_SEQ;
    return -1;
  }
  const long long pos = a.positions[n];
  if (pos < 0 || pos >= (long long)a.max_blocks * a.bs) {
    flag = DA_DEV_BAD_SEQ_LEN;
    return -1;
  }
  const int blk = a.block_table[(long long)seq * a.max_blocks + pos / a.bs];
  if (blk < 0 || blk >= a.num_blocks) {
    flag = DA_DEV_BAD_BLOCK;
    return -1;
  }
  return (long long)blk * a.bs + pos % a.bs;
}

// Minimum and maximum that a NaN wins.
__device__ __forceinline__ float min_nan(float x, float y) {
  float z;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

// Least and largest of eight values.
__device__ __forceinline__ float2 extent8(const float (&x)[8]) {
  float2 e = make_float2(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) e = make_float2(min_nan(e.x, x[i]), max_nan(e.y, x[i]));
  return e;
}

// Scale and zero of a group with this extent, as they are stored and as f32.  The extent is
// taken to f16's range first, so that both are finite but for a NaN.
struct Q4Param {
  uint32_t word;
  float scale, zero, inv;  // inv: 1 / scale to 2^-22
};
__device__ __forceinline__ Q4Param q4_param(float2 e) {
  const float lo = max_nan(min_nan(e.x, 65504.f), -65504.f);
  const float hi = max_nan(min_nan(e.y, 65504.f), -65504.f);
  const __half z = __float2half_rn(lo), s = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
  Q4Param p;
  p.word = (uint32_t)__half_as_ushort(s) | (uint32_t)__half_as_ushort(z) << 16;
  p.scale = __half2float(s);
  p.zero = __half2float(z);
  p.inv = __fdividef(1.f, p.scale);
  return p;
}

// Eight codes: round((x - zero) / scale), ties to even, within 0..15; 0 without a scale.  The quotient by
// the reciprocal (good to 2^-22, its product to 2^-24) is off from the rounded one by 15.5 * 1.5 * 2^-22 at most, 6e-6, so
// it says the code of any value that is not that near to the middle between two; where one is (a value in
// 50,000), the eight are divided.  (Divided always, 12,287 tokens
// x 16 rows x 128 took 58 us, where this took 39.)
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[8], const Q4Param& p) {
  if (!(p.scale > 0.f)) return 0;
  // 1.5 * 2^23: added to a small number, its last bits are the number's nearest integer
  const float2 kInt = make_float2(12582912.f, 12582912.f), kBack = make_float2(-12582912.f, -12582912.f);
  const float2 minus = make_float2(-p.zero, -p.zero), inv = make_float2(p.inv, p.inv);
  uint32_t w = 0;
  float far = 0.f;  // from the nearest integer
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    float2 q = da::mul2(da::add2(make_float2(x[i], x[i + 1]), minus), inv);
    q = make_float2(fminf(fmaxf(q.x, 0.f), 15.f), fminf(fmaxf(q.y, 0.f), 15.f));
    const float2 t = da::add2(q, kInt), c = da::add2(t, kBack);
    far = fmaxf(far, fmaxf(fabsf(q.x - c.x), fabsf(q.y - c.y)));
    w = (w * 16 + __float_as_uint(t.y)) * 16 + __float_as_uint(t.x);
  }
  // the numbers' upper bits, 0x4b400000, in every one of the eight places
  w -= 0x4b400000u * 0x11111111u;
  if (far > 0.5f - 1e-5f) {
    w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(fmaxf(rintf(__fdiv_rn(x[i] - p.zero, p.scale)), 0.f), 15.f);
      w |= (uint32_t)c << (4 * i);
    }
  }
  return w;
}

template <typename T, int D, bool IL, int MODE>
__global__ void __launch_bounds__(kRopeThreads, rope_ctas(MODE)) rope_kernel(const RopeArgs a) {
  constexpr bool APPEND = MODE != kNormRope;
  constexpr int TPR = D / 16;                 // threads of a row
  constexpr int RPI = kRopeThreads / TPR;     // rows of a round
  // cosine and sine of pairs 2j and 2j + 1 of chunk c at [j][c]: a row's threads read
  // neighbouring 16 bytes (in the order of the pairs, four of them met in one bank: 92 us against
  // 83 on the case above)
  __shared__ float4 cs[max_tokens(MODE)][4][TPR];
  __shared__ long long place[max_tokens(MODE)];     // append: row of the pool, or one of:
  constexpr long long kDropped = -1, kPadding = -2;
  // append in 4 bits: extents of the chunks of the rows in work
  __shared__ float4 extent[MODE == kAppendQ4 ? RPI : 1][D / 16];
  const int n0 = blockIdx.x * a.tokens, tokens = min(a.tokens, a.N - n0);
  const int c = threadIdx.x % TPR;
  const int nrot = a.rd / 16;  // chunk pairs that are rotated
  const bool rot = c < nrot;
  const int lo = IL ? 16 * c : rot ? 8 * c : a.rd + 16 * (c - nrot);
  const int hi = (IL || !rot) ? lo + 8 : a.rd / 2 + 8 * c;
  const int rows = tokens * a.heads;
  da::let_next_grid_start();
  da::wait_for_grid_before();

  struct Row {
    int t, h, kind;  // token of the CTA, head, 0 q / 1 k / 2 v
    Raw<T> lo, hi;
  };
  auto fetch = [&](int r) {
    Row x;
    x.t = (int)(((uint64_t)r * a.inv_heads) >> 32);
    x.h = r - x.t * a.heads;
    x.kind = x.h < a.Hq ? 0 : x.h < a.Hq + a.Hk ? 1 : 2;
    x.h -= x.kind == 0 ? 0 : x.kind == 1 ? a.Hq : a.Hq + a.Hk;
    const long long n = n0 + x.t;
    const T* src;
    if constexpr (MODE == kAppendQ4) {
      const void* from = x.kind == 0 ? a.q : x.kind == 1 ? a.k : a.v;
      const long long ts = x.kind == 0 ? a.q_ts : x.kind == 1 ? a.k_ts : a.v_ts;
      const long long hs = x.kind == 0 ? a.q_hs : x.kind == 1 ? a.k_hs : a.v_hs;
      src = static_cast<const T*>(from) + n * ts + x.h * hs;
    } else {  // an address of each: with selected terms the f32 norm and rotation spills 24 bytes more, 41 for 28.8 us
      src = x.kind == 0   ? static_cast<const T*>(a.q) + n * a.q_ts + x.h * a.q_hs
            : x.kind == 1 ? static_cast<const T*>(a.k) + n * a.k_ts + x.h * a.k_hs
                          : static_cast<const T*>(a.v) + n * a.v_ts + x.h * a.v_hs;
    }
    x.lo = load8(src + lo);
    x.hi = load8(src + hi);
    return x;
  };
  int r = threadIdx.x / TPR;
  Row next = fetch(min(r, rows - 1));  // rows past the last are loaded, not stored

  for (int i = threadIdx.x; i < tokens * (a.rd / 2); i += kRopeThreads) {
    const int t = i / (a.rd / 2), f = i - t * (a.rd / 2);
    const uint64_t turns = (uint64_t)(long long)a.positions[n0 + t] * a.freqs[f];
    // quarter turns, and the rest in [-1/8, 1/8) turns: rounded to f32 as a small number
    const uint64_t quarter = (turns + (1ull << 61)) >> 62;
    const float half_turns = __ll2float_rn((long long)(turns - (quarter << 62))) * 0x1p-63f;
    float sn, cn;
    sincospif(half_turns, &sn, &cn);
    const float x = quarter & 1 ? -sn : cn, y = quarter & 1 ? cn : sn;
    float2* at = reinterpret_cast<float2*>(&cs[t][f % 8 / 2][f / 8]) + f % 2;
    *at = quarter & 2 ? make_float2(-x, -y) : make_float2(x, y);
  }
  if constexpr (APPEND) {
    if ((int)threadIdx.x < tokens) {
      int flag;
      bool pad;
      const long long row = cache_row(a, n0 + threadIdx.x, flag, pad);
      long long at = row;
      if constexpr (MODE == kAppendQ4)  // its page's first byte, and its row there
        at = ((row >> a.log2_bs) * a.Hkv * a.page_bytes) << 8 | (row & (a.bs - 1));
      place[threadIdx.x] = pad ? kPadding : flag ? kDropped : at;
      if (flag && a.dev_status) atomicOr(a.dev_status, flag);
    }
  }
  __syncthreads();

  float g[2][8];  // the weights of q or k
  int have = -1;
  // a warp's threads run the same number of rounds: the norm's sum is taken across them
  for (int r0 = 0; r0 < rows; r0 += RPI, r += RPI) {
    const Row cur = next;
    if (r0 + RPI < rows) next = fetch(min(r + RPI, rows - 1));
    float x[2][8];
    values8(cur.lo, x[0]);
    values8(cur.hi, x[1]);
    if (a.norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[0][i], x[0][i], fmaf(x[1][i], x[1][i], ss));
#pragma unroll
      for (int o = TPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (cur.kind < 2) {
        const float m = 1.f / sqrtf(ss * (1.f / D) + a.eps);
        const float* w = cur.kind == 0 ? a.qw : a.kw;
        if (w && cur.kind != have) {
          values8(load8(w + lo), g[0]);
          values8(load8(w + hi), g[1]);
          have = cur.kind;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[0][i] *= w ? m * (g[0][i] + a.woff) : m;
          x[1][i] *= w ? m * (g[1][i] + a.woff) : m;
        }
      }
    }
    if (MODE != kAppendQ4 && r >= rows) continue;
    if (rot && cur.kind < 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 two = cs[cur.t][i / 2][c];
        const float2 t = i % 2 ? make_float2(two.z, two.w) : make_float2(two.x, two.y);
        float& y0 = IL ? x[i / 4][2 * (i % 4)] : x[0][i];
        float& y1 = IL ? x[i / 4][2 * (i % 4) + 1] : x[1][i];
        const float z0 = y0 * t.x - y1 * t.y;
        y1 = y0 * t.y + y1 * t.x;
        y0 = z0;
      }
    }
    long long row = 0;
    if constexpr (APPEND) row = place[cur.t];
    if constexpr (MODE == kAppendQ4) {
      // A group's chunks are in several threads.  Where a thread's two are neighbours, their extents go by
      // shuffles; else the rotation gives the order: each thread puts its chunks' extents down,
      // and takes those of the groups that they belong to.
      float2* ext = reinterpret_cast<float2*>(extent[threadIdx.x / TPR]);
      const bool side_by_side = IL || a.rd == 0;
      float2 own = extent8(x[0]);
      {
        const float2 e = extent8(x[1]);
        if (side_by_side) {
          own = make_float2(min_nan(own.x, e.x), max_nan(own.y, e.y));
          for (int by = 1; by < 1 << (a.log2_group - 4); by <<= 1)
            own = make_float2(min_nan(own.x, __shfl_xor_sync(0xffffffffu, own.x, by)),
                              max_nan(own.y, __shfl_xor_sync(0xffffffffu, own.y, by)));
        } else {
          __syncwarp();
          ext[lo / 8] = own;
          ext[hi / 8] = e;
          __syncwarp();
        }
      }
      const bool kept = r < rows && cur.kind != 0 && row >= 0;
      uint8_t* page = nullptr;
      int t = 0, words = 0;
      if (kept) {
        t = (int)(row & 255);
        page = a.q4_pool + (row >> 8) + cur.h * (int)a.page_bytes;
        words = D >> a.log2_group;  // params of a row
      }
      Q4Param p;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int d = half ? hi : lo, g = d & -(1 << a.log2_group);
        if (!side_by_side) {
          float2 e = make_float2(INFINITY, -INFINITY);
          for (int i = 0; i < 1 << (a.log2_group - 4); ++i) {
            const float4 two = extent[threadIdx.x / TPR][g / 16 + i];
            e = make_float2(min_nan(e.x, min_nan(two.x, two.z)), max_nan(e.y, max_nan(two.y, two.w)));
          }
          p = q4_param(e);
        } else if (half == 0) {
          p = q4_param(own);
        }
        if (!kept) continue;
        uint8_t* codes = page + (cur.kind == 2 ? a.bs * (D / 2) : 0) + t * (D / 2);
        const int piece = (d / 32) ^ da::piece_xor<D>(t);
        *reinterpret_cast<uint32_t*>(codes + 16 * piece + d % 32 / 2) = q4_codes(x[half], p);
        if (d == g)
          reinterpret_cast<uint32_t*>(page + a.bs * D)[((cur.kind == 2 ? a.bs : 0) + t) * words +
                                                       (g >> a.log2_group)] = p.word;
      }
      if (cur.kind != 0 || r >= rows) continue;
    }
    if (cur.kind == 0) {
      if (APPEND && row == kPadding) continue;
      float* dst = a.q_out + ((long long)(n0 + cur.t) * a.Hq + cur.h) * D;
      store8(dst + lo, x[0], a.wide_out);
      store8(dst + hi, x[1], a.wide_out);
    } else {
      uint16_t* dst;
      if constexpr (MODE == kAppendQ4) {
        continue;  // done above
      } else if constexpr (APPEND) {
        if (row < 0) continue;
        dst = (cur.kind == 2 ? a.v_pool : a.k_pool) + (row * a.Hkv + cur.h) * D;
      } else {
        dst = a.k_out + ((long long)(n0 + cur.t) * a.Hkv + cur.h) * D;
      }
      store8(dst + lo, x[0]);
      store8(dst + hi, x[1]);
    }
  }
}

template <typename T, int D, int MODE>
cudaError_t launch_rope_d(const RopeArgs& a, int il, cudaStream_t s) {
  const int grid = (a.N + a.tokens - 1) / a.tokens;
  return da::launch_early(il ? rope_kernel<T, D, true, MODE> : rope_kernel<T, D, false, MODE>,
                          grid, kRopeThreads, 0, s, a);
}

template <typename T, int MODE>
cudaError_t launch_rope_t(const RopeArgs& a, int D, int il, cudaStream_t s) {
  if (D == 64) return launch_rope_d<T, 64, MODE>(a, il, s);
  if (D == 128) return launch_rope_d<T, 128, MODE>(a, il, s);
  return launch_rope_d<T, 256, MODE>(a, il, s);
}

template <int MODE>
int launch_rope(RopeArgs& a, const da_rope_params* r, int D, int num_tokens, void* stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.N = num_tokens;
  a.heads = a.Hq + a.Hk + (MODE != kNormRope ? a.Hkv : 0);
  a.inv_heads = (0x100000000ULL + a.heads - 1) / a.heads;
  // Tokens of a CTA: the fewest waves of CTAs that hold them, and so many that these waves are
  // filled but for what rounding to whole tokens leaves (12,287 tokens: 11 each, 1117 of 1216 places).
  int sms = 0;
  const int st = da::device_sms(&sms);
  if (st != DA_OK) return st;
  const int wave = sms * rope_ctas(MODE);  // CTAs that run at once
  const int waves = (num_tokens - 1) / (wave * max_tokens(MODE)) + 1;
  a.tokens = (num_tokens - 1) / (wave * waves) + 1;
  const cudaError_t err =
      r->type == DA_TYPE_F32   ? launch_rope_t<float, MODE>(a, D, r->interleaved, s)
      : r->type == DA_TYPE_F16 ? launch_rope_t<__half, MODE>(a, D, r->interleaved, s)
                               : launch_rope_t<__nv_bfloat16, MODE>(a, D, r->interleaved, s);
  return err == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A strided input: every row on a 16-byte boundary, offsets within 63 bits.
int check_rows(const void* p, long long ts, long long hs, int esize, int tokens, int heads) {
  if (!aligned(p, 16) || ts < 0 || hs < 0) return DA_ERR_INVALID;
  if ((ts * esize) % 16 != 0 || (hs * esize) % 16 != 0) return DA_ERR_INVALID;
  const long long lim = 1LL << 40;  // elements between rows: far past any device's memory
  if (ts > lim || hs > lim || tokens < 0 || heads <= 0) return DA_ERR_INVALID;
  return DA_OK;
}

int check_rope(const da_rope_params* r, int D) {
  if (!r) return DA_ERR_INVALID;
  if (r->type != DA_TYPE_F32 && r->type != DA_TYPE_F16 && r->type != DA_TYPE_BF16)
    return DA_ERR_INVALID;
  if (D <= 0) return DA_ERR_INVALID;
  if (D != 64 && D != 128 && D != 256) return DA_ERR_UNSUPPORTED;
  if (r->rotary_dim < 0 || r->rotary_dim > D || r->rotary_dim % 2 != 0) return DA_ERR_INVALID;
  if (r->rotary_dim % 16 != 0) return DA_ERR_UNSUPPORTED;
  if ((r->interleaved != 0 && r->interleaved != 1) || (r->norm != 0 && r->norm != 1))
    return DA_ERR_INVALID;
  if (r->norm && (!(r->eps >= 0.f) || isinf(r->eps) || !isfinite(r->weight_offset)))
    return DA_ERR_INVALID;
  if (r->rotary_dim > 0 && (!r->freqs || !aligned(r->freqs, 8))) return DA_ERR_INVALID;
  if (r->norm && ((r->q_weight && !aligned(r->q_weight, 16)) ||
                  (r->k_weight && !aligned(r->k_weight, 16))))
    return DA_ERR_INVALID;
  return DA_OK;
}

void fill_args(RopeArgs& a, const da_rope_params* r, const void* q, const void* k,
               const int32_t* positions, int Hq, int Hkv, float* q_out) {
  a.q = q;
  a.k = k;
  a.q_ts = r->q_token_stride;
  a.q_hs = r->q_head_stride;
  a.k_ts = r->k_token_stride;
  a.k_hs = r->k_head_stride;
  a.v_ts = r->v_token_stride;
  a.v_hs = r->v_head_stride;
  a.qw = r->norm ? r->q_weight : nullptr;
  a.kw = r->norm ? r->k_weight : nullptr;
  a.freqs = r->freqs;
  a.positions = positions;
  a.Hq = q ? Hq : 0;
  a.Hk = k ? Hkv : 0;
  a.Hkv = Hkv;
  a.rd = r->rotary_dim;
  a.norm = r->norm;
  a.eps = r->eps;
  a.woff = r->weight_offset;
  a.q_out = q_out;
  a.wide_out = aligned(q_out, 32);
}

// Checks of an append, and its arguments but for where it writes (k_to, v_to are only checked).
int append_args(RopeArgs& a, const da_params* p, const da_rope_params* r, int32_t num_tokens,
                const void* q, const void* k_new, const void* v_new, const int32_t* positions,
                const int32_t* token_seq, const int32_t* block_table, float* q_out,
                int32_t* dev_status, const void* k_to, const void* v_to) {
  int st = da::check_append_params(p);
  if (st != DA_OK) return st;
  st = check_rope(r, p->head_dim);
  if (st != DA_OK) return st;
  if (num_tokens < 0 || (!token_seq && num_tokens != p->batch)) return DA_ERR_INVALID;
  if (!k_new || !v_new || !positions || !block_table || !k_to || !v_to) return DA_ERR_INVALID;
  if ((q == nullptr) != (q_out == nullptr)) return DA_ERR_INVALID;
  if (!aligned(k_to, 16) || !aligned(v_to, 16) || !aligned(positions, 4) ||
      !aligned(block_table, 4) || (token_seq && !aligned(token_seq, 4)) ||
      (dev_status && !aligned(dev_status, 4)) || (q_out && !aligned(q_out, 16)))
    return DA_ERR_INVALID;
  const int esize = r->type == DA_TYPE_F32 ? 4 : 2;
  st = check_rows(k_new, r->k_token_stride, r->k_head_stride, esize, num_tokens, p->num_kv_heads);
  if (st != DA_OK) return st;
  st = check_rows(v_new, r->v_token_stride, r->v_head_stride, esize, num_tokens, p->num_kv_heads);
  if (st != DA_OK) return st;
  if (q) {
    st = check_rows(q, r->q_token_stride, r->q_head_stride, esize, num_tokens, p->num_q_heads);
    if (st != DA_OK) return st;
  }
  if ((long long)(q ? p->num_q_heads : 0) + 2LL * p->num_kv_heads > 4096)
    return DA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return DA_OK;
  fill_args(a, r, q, k_new, positions, p->num_q_heads, p->num_kv_heads, q_out);
  a.v = v_new;
  a.token_seq = token_seq;
  a.block_table = block_table;
  a.batch = p->batch;
  a.bs = p->block_size;
  a.max_blocks = p->max_blocks_per_seq;
  a.num_blocks = p->num_blocks;
  a.dev_status = dev_status;
  return DA_OK;
}

}  // namespace

extern "C" {

int decode_attn_rope_freqs(int32_t rotary_dim, double theta, const double* inv_freq,
                           uint64_t* freqs) {
  if (rotary_dim < 0 || rotary_dim % 2 != 0 || (rotary_dim > 0 && !freqs)) return DA_ERR_INVALID;
  if (!inv_freq && !(theta > 0.0 && isfinite(theta))) return DA_ERR_INVALID;
  auto radians = [&](int i) { return inv_freq ? inv_freq[i] : pow(theta, -2.0 * i / rotary_dim); };
  for (int i = 0; i < rotary_dim / 2; ++i)
    if (!isfinite(radians(i))) return DA_ERR_INVALID;  // a power may overflow too
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double w = radians(i);
    // the fraction of a turn, in [0, 1); whole turns a position drop out
    double t = w / 6.283185307179586476925286766559;
    t -= floor(t);
    const double u = rint(t * 18446744073709551616.0);
    freqs[i] = u >= 18446744073709551616.0 ? 0 : (uint64_t)u;
  }
  return DA_OK;
}

int decode_attn_qk_norm_rope(const da_rope_params* r, int32_t num_tokens, int32_t num_q_heads,
                             int32_t num_kv_heads, int32_t head_dim, const void* q, const void* k,
                             const int32_t* positions, float* q_out, uint16_t* k_out,
                             void* stream) {
  int st = check_rope(r, head_dim);
  if (st != DA_OK) return st;
  if (num_tokens < 0 || (!q && !k)) return DA_ERR_INVALID;
  const int esize = r->type == DA_TYPE_F32 ? 4 : 2;
  if (q) {
    if (!q_out || !aligned(q_out, 16)) return DA_ERR_INVALID;
    st = check_rows(q, r->q_token_stride, r->q_head_stride, esize, num_tokens, num_q_heads);
    if (st != DA_OK) return st;
  }
  if (k) {
    if (!k_out || !aligned(k_out, 16)) return DA_ERR_INVALID;
    st = check_rows(k, r->k_token_stride, r->k_head_stride, esize, num_tokens, num_kv_heads);
    if (st != DA_OK) return st;
  }
  if ((long long)(q ? num_q_heads : 0) + (k ? num_kv_heads : 0) > 4096) return DA_ERR_UNSUPPORTED;
  if (r->rotary_dim > 0 && !positions) return DA_ERR_INVALID;
  if (positions && !aligned(positions, 4)) return DA_ERR_INVALID;
  if (num_tokens == 0) return DA_OK;
  RopeArgs a = {};
  fill_args(a, r, q, k, positions, num_q_heads, num_kv_heads, q_out);
  a.k_out = k_out;
  return launch_rope<kNormRope>(a, r, head_dim, num_tokens, stream);
}

int decode_attn_append_paged_rope(const da_params* p, const da_rope_params* r, int32_t num_tokens,
                                  const void* q, const void* k_new, const void* v_new,
                                  const int32_t* positions, const int32_t* token_seq,
                                  const int32_t* block_table, float* q_out, uint16_t* k_pool,
                                  uint16_t* v_pool, int32_t* dev_status, void* stream) {
  RopeArgs a = {};
  const int st = append_args(a, p, r, num_tokens, q, k_new, v_new, positions, token_seq,
                             block_table, q_out, dev_status, k_pool, v_pool);
  if (st != DA_OK || num_tokens == 0) return st;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  return launch_rope<kAppend>(a, r, p->head_dim, num_tokens, stream);
}

int decode_attn_append_paged_q4(const da_params* p, const da_rope_params* r, int32_t group,
                                int32_t num_tokens, const void* q, const void* k_new,
                                const void* v_new, const int32_t* positions,
                                const int32_t* token_seq, const int32_t* block_table,
                                float* q_out, uint8_t* pool, int32_t* dev_status, void* stream) {
  int st = da::check_append_params(p);
  if (st == DA_OK) st = da::check_q4(p, group);
  if (st != DA_OK) return st;
  RopeArgs a = {};
  st = append_args(a, p, r, num_tokens, q, k_new, v_new, positions, token_seq, block_table, q_out,
                   dev_status, pool, pool);
  if (st != DA_OK || num_tokens == 0) return st;
  a.q4_pool = pool;
  while ((1 << a.log2_group) < group) ++a.log2_group;
  while ((1 << a.log2_bs) < p->block_size) ++a.log2_bs;
  a.page_bytes = da::q4_page_bytes(p->block_size, p->head_dim, group);
  return launch_rope<kAppendQ4>(a, r, p->head_dim, num_tokens, stream);
}

}  // extern "C"
