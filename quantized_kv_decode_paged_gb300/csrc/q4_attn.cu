// q4_attn.cu — decode attention over a paged cache held in 4 bits.
//
// Mathematics.  With q in base-2 units (scale * log2(e)), a score is
//   s_t = sum_g scale_tg sum_{d in g} q_d code_td + zero_tg sum_{d in g} q_d
// over the groups g of a key's row, or with code - 8 and zero + 8 scale in place of the two, and for the
// value groups alike
//   out_d = (sum_t (p_t scale_tg) (code_td - 8) + sum_t p_t (zero_tg + 8 scale_tg)) / sum_t p_t:
// codes enter the products as they are and the scales go into scores and weights.  (Without the 8
// the codes' common part, 7.5 sum p scale, grows with the keys, the rest with their root, and the
// sums would lose what lies between.)
//
// Codes as f16 operands.  A nibble with zeros around it is, read as an f16 subnormal, code * 2^-24, or
// code * 2^-20 one nibble further up; one fused multiply-add makes it (code - 8) 2^-9, exactly.  Eight
// codes take a shift, four ANDs and four of those.  (The subnormals themselves as operands: their
// products are exact too, but are lined up by the exponent that they do not have, and the sums lost up to 7
// more bits: 1e-5 of the result.)
//
// Precision.  Q and the weights are two f16 terms each (22 bits), the row's largest value of Q scaled
// to 2^14.  A weight times the value scale stays inside f16: the reference m of a row is
// taken over s_t + e_t, e_t the exponent of the key's largest value scale, and p_t = 2^(s_t - m + 10), so
// p_t scale_tg is at most 2^15 (m moves when some s_t + e_t passes it by 5), and lies 34 powers of two above
// f16's smallest step at m.  mma.sync adds with truncation, so a sum takes at most kChain steps and is then
// added up in f32.
//
// Work.  A unit is (sequence, kv head, up to 64 query rows: query tokens x heads of the kv head), a tile 128
// of its keys.  The tiles of all units are cut into equal shares, one a CTA; a unit that two CTAs share
// leaves its parts' states in the workspace, which q4_merge_kernel adds up.  A producer warp copies pages (one
// bulk copy a page of a head, which holds codes and scales of keys and values) into a ring of tiles;
// eight consumer warps take 16 keys x 8 rows at a time: S^T = K Q^T and O^T += V^T P^T with
// mma.m16n8k16, keys and value columns as M, so that 8 rows of Q fill N.  The row order of the
// 16 keys (tau below) is such that the fragments of K by ldmatrix and of V by its transposing byte form meet
// in one layout and no bank twice.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "../../include/decode_attn.h"
#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace {

constexpr int kWarps = 8;               // consumer warps
constexpr int kThreads = 32 * (kWarps + 4);  // and a warpgroup of which one warp copies
// Registers of a thread of the two kinds: 2 * 232 + 40 = 3 * 168, what the launch has.
constexpr int kConsumerRegs = 232, kProducerRegs = 40;
constexpr int kTok = 16 * kWarps;       // keys of a tile
constexpr int kRows = 8;                // query rows of a warp
constexpr int kMaxGroups = kWarps;      // groups of kRows rows of a unit
constexpr int kMaxBatch = 1024;         // sequences of a launch
constexpr int kChain = 4;               // steps of 16 keys between f32 additions
constexpr float kShift = 10.f, kSlack = 5.f;
constexpr float kLn2 = 0.6931471805599453f;

struct Q4Params {
  const float* q;
  const uint8_t* pool;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* q_pos;
  float* out;
  float* lse;
  int32_t* dev_status;
  int B, T, G, R, Hq, Hkv, log2_bs, max_blocks, num_blocks, window, causal;
  int groups, blocks;  // row groups of a unit (a power of two), units of a kv head
  int units;           // of the batch; stages of the ring
  int split, stages, log2_eb;  // eb: rows of a page's piece in a tile, min(block size, kTok)
  float qscale, softcap2, softcap_inv;
  long long page_bytes;
  unsigned long long wait_ns;
  int test_skip_arm;
  // workspace
  int4* desc;      // [CTAs] of the unit that is cut at the CTA's end: b (or -1), unit, slot, last CTA
  float2* part_ml;  // [CTAs][2][groups * 8]: reference and sum
  float* part_o;    // [CTAs][2][groups * 8][D]
};

// ------------------------------------------------------------------ what a sequence sees
struct Seq {
  int len, lo, hi;  // keys [lo, hi) are seen by some row
  int qp;           // position of query token 0
  int tile0, tiles;
};

__device__ __forceinline__ int seq_info(const Q4Params& p, int b, Seq& s) {
  int flags = 0;
  const long long cap = (long long)p.max_blocks << p.log2_bs;
  long long len = p.seq_lens[b];
  if (len < 0 || len > cap) {
    flags = DA_DEV_BAD_SEQ_LEN;
    len = len < 0 ? 0 : cap;
  }
  long long qp = len - p.T;
  bool none = len == 0;
  if (p.q_pos) {
    qp = p.q_pos[b];
    if (qp < 0) flags |= DA_DEV_BAD_QPOS, none = true;
  }
  long long lo = p.window > 0 && qp >= p.window ? qp - p.window + 1 : 0;
  long long hi = p.causal && qp + p.T < len ? qp + p.T : len;
  if (none || hi <= lo) lo = hi = 0;
  s.len = (int)len;
  s.lo = (int)lo;
  s.hi = (int)hi;
  s.qp = (int)(qp < 0x7fff0000 ? qp : 0x7fff0000);  // past every key and window alike
  s.tile0 = (int)(lo / kTok);
  s.tiles = hi > lo ? (int)((hi + kTok - 1) / kTok) - s.tile0 : 0;
  return flags;
}

// Keys [lo, hi) that query token t sees.
__device__ __forceinline__ void row_keys(const Q4Params& p, const Seq& s, int t, int& lo, int& hi) {
  const long long qp = (long long)s.qp + t;
  lo = p.window > 0 && qp >= p.window ? (int)(qp - p.window + 1) : 0;
  hi = p.causal && qp + 1 < s.len ? (int)(qp + 1) : s.len;
  if (s.tiles == 0) hi = lo;
}

__device__ __forceinline__ int share_start(int cta, int total, int grid) {
  return (int)((long long)cta * total / grid);
}

// A CTA's part of a unit.
struct Seg {
  int b, kv, block;  // block of row groups
  int i0, i1;        // tiles [i0, i1) of the sequence's
  int slot;          // -1: the whole unit; else its place among the CTA's states
};

struct Walk {
  int g, end, n, b;  // next tile and end of the share, segments so far, last sequence
  int upb;           // units of a sequence
};

struct Shared {
  uint64_t full[16], empty[16];
  uint32_t bad[16];  // pages of a stage's tile that are outside the pool
  float2 ml[kWarps][kRows];
  int warp_sum[kThreads / 32];
  int abort, flags;
};

// Next segment of this CTA; false at its end.  pre: tiles of the sequences before each.
__device__ __forceinline__ bool next_seg(const Q4Params& p, const int* pre, Walk& w, Seg& s) {
  int unit;
  if (p.split) {
    if (w.g >= w.end) return false;
    while ((long long)pre[w.b + 1] * w.upb <= w.g) ++w.b;
    const int nt = pre[w.b + 1] - pre[w.b], rel = w.g - pre[w.b] * w.upb;
    unit = rel / nt;
    s.i0 = rel - unit * nt;
    s.i1 = min(nt, s.i0 + (w.end - w.g));
    s.slot = s.i0 == 0 && s.i1 == nt ? -1 : w.n ? 1 : 0;
    w.g += s.i1 - s.i0;
    s.b = w.b;
  } else {
    const int u = blockIdx.x + w.n * gridDim.x;
    if (u >= p.units) return false;
    s.b = u / w.upb;
    unit = u - s.b * w.upb;
    s.i0 = 0;
    s.i1 = -1;  // all of the sequence's
    s.slot = -1;
  }
  ++w.n;
  s.kv = unit / p.blocks;
  s.block = unit - s.kv * p.blocks;
  return true;
}

// ------------------------------------------------------------------ waits
// A wait that runs out sets the abort flag: later waits return at once, no more copies are made, and
// every warp runs its loops to the end on whatever shared memory holds.
__device__ __forceinline__ bool wait_for(const Q4Params& p, Shared& sh, uint64_t* bar,
                                         uint32_t parity) {
  if (*(volatile int*)&sh.abort) return false;
  if (da::mbar_wait(bar, parity, &sh.abort, p.wait_ns)) return true;
  *(volatile int*)&sh.abort = 1;
  return false;
}

// ------------------------------------------------------------------ arithmetic
// cap * tanh(y) in base-2 units: below |y| = 1/2 the polynomial of prefix_attn.cu's cap_near, above it
// the identity in 2^x.
__device__ __forceinline__ float soft_cap(float y, float cap2) {
  const float t = y * y, z = y * cap2;
  float c = fmaf(0.017241476f, t, -0.053045485f);
  c = fmaf(c, t, 0.13325879f);
  c = fmaf(c, t, -0.33333144f);
  const float small = fmaf(z, t * c, z);
  const float big = cap2 * (1.f - __fdividef(2.f, da::ex2_ftz(y * 2.8853900817779268f) + 1.f));
  return fabsf(y) <= 0.5f ? small : big;
}

__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float half_lo(uint32_t w) {
  return __half2float(__ushort_as_half((unsigned short)w));
}
__device__ __forceinline__ float half_hi(uint32_t w) {
  return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}

// The codes of a byte pair's low or high nibbles as (code - 8) 2^-9.
__device__ __forceinline__ uint32_t codes2(uint32_t w, bool high) {
  uint32_t z;
  asm("fma.rn.f16x2 %0, %1, %2, %3;"
      : "=r"(z)
      : "r"(w & (high ? 0x00f000f0u : 0x000f000fu)),  // 2^-20, 2^-24
        "r"(high ? 0x68006800u : 0x78007800u),        // 2^11, 2^15
        "r"(0xa400a400u));                            // -2^-6
  return z;
}

template <int D, int NG>
struct Geo {
  static constexpr int P = D / 32;       // 16-byte pieces of a row
  static constexpr int GP = P / NG;      // pieces of a group
  static constexpr int RB = D / 2;       // bytes of a row's codes
  static constexpr int ROW = D + 8 * NG;  // bytes of a key's and a value's row
  static constexpr int STAGE = kTok * ROW;
  static constexpr bool QREG = D <= 128;  // Q's fragments in registers, else in shared memory
  static constexpr int COL = D + 4;       // floats between rows of a state in shared memory
  static constexpr int QBYTES = QREG ? 0 : kMaxGroups * P * 2 * 512;
  static constexpr int OBYTES = kWarps * kRows * COL * 4;
  static constexpr int UNION = QBYTES > OBYTES ? QBYTES : OBYTES;
};

template <int D, int NG>
__global__ void __launch_bounds__(kThreads, 1) q4_kernel(const __grid_constant__ Q4Params p) {
  using g_ = Geo<D, NG>;
  constexpr int P = g_::P, GP = g_::GP, RB = g_::RB, MT = 2 * P;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Shared sh;
  uint8_t* ring = dyn;
  uint8_t* scratch = dyn + (size_t)p.stages * g_::STAGE;  // Q's fragments, states
  int* pre = reinterpret_cast<int*>(scratch + g_::UNION);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int eb = 1 << p.log2_eb, bs = 1 << p.log2_bs;
  const int rec = eb * g_::ROW;  // bytes of a page's piece in a tile

  if (tid == 0) {
    sh.abort = sh.flags = 0;
    for (int i = 0; i < p.stages; ++i) {
      da::mbar_init(&sh.full[i], 1);
      da::mbar_init(&sh.empty[i], kWarps);
    }
    da::fence_mbarrier_init();
  }
  da::wait_for_grid_before();
  da::let_next_grid_start();

  Walk walk;
  walk.upb = p.Hkv * p.blocks;
  walk.n = 0;
  walk.g = walk.end = walk.b = 0;
  int total = 0, shares = 0;  // tiles, CTAs that have some: at least one each
  if (p.split) {
    // tiles of the sequences before each
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(tid * per, p.B);
    const int b1 = min(b0 + per, p.B);
    int mine = 0, bad = 0;
    for (int b = b0; b < b1; ++b) {
      Seq s;
      bad |= seq_info(p, b, s);
      pre[b + 1] = s.tiles;
      mine += s.tiles;
    }
    if (bad && blockIdx.x == 0 && p.dev_status) atomicOr(p.dev_status, bad);
    int upto = mine;
#pragma unroll
    for (int by = 1; by < 32; by <<= 1) {
      const int below = __shfl_up_sync(0xffffffffu, upto, by);
      if (lane >= by) upto += below;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncthreads();
    int run = upto - mine;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) run += sh.warp_sum[i];
      total += sh.warp_sum[i];
    }
    for (int b = b0; b < b1; ++b) run += pre[b + 1], pre[b + 1] = run;
    if (tid == 0) pre[0] = 0;
    total *= walk.upb;
    __syncthreads();
    shares = min((int)gridDim.x, total);
    if ((int)blockIdx.x < shares) {
      walk.g = share_start(blockIdx.x, total, shares);
      walk.end = share_start(blockIdx.x + 1, total, shares);
      int lo = 0, hi = p.B;  // the sequence that holds the first tile
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if ((long long)pre[mid] * walk.upb <= walk.g) lo = mid;
        else hi = mid;
      }
      walk.b = lo;
    }
  } else {
    __syncthreads();
  }

  if (warp >= kWarps) {
    // ---------------------------------------------------------------- producer
    da::setmaxnreg_dec<kProducerRegs>();
    if (warp == kWarps) {
    Seg sg;
    int stage = 0, round = 0;
    bool skip = p.test_skip_arm && blockIdx.x == 0;
    const int pieces = kTok >> p.log2_eb;
    bool went = true;
    while (went && next_seg(p, pre, walk, sg)) {
      Seq s;
      const int bad = seq_info(p, sg.b, s);
      if (!p.split && bad && lane == 0 && p.dev_status) atomicOr(p.dev_status, bad);
      const int end = sg.i1 < 0 ? s.tiles : sg.i1;
      auto block_id = [&](int i) {  // of this lane's piece of tile i; -1: not read, -2: outside
        const int k = (s.tile0 + i) * kTok + (lane << p.log2_eb);
        if (i >= end || lane >= pieces || k >= s.hi || k + eb <= s.lo) return -1;
        const int id = p.table[(long long)sg.b * p.max_blocks + (k >> p.log2_bs)];
        return id >= 0 && id < p.num_blocks ? id : -2;
      };
      int id = block_id(sg.i0);
      for (int i = sg.i0; i < end; ++i) {
        const int now = id;
        id = block_id(i + 1);
        const uint32_t bad_pages = __ballot_sync(0xffffffffu, now == -2);
        const uint32_t pages = __ballot_sync(0xffffffffu, now >= 0);
        if (bad_pages && lane == 0 && p.dev_status) atomicOr(p.dev_status, DA_DEV_BAD_BLOCK);
        if (round > 0)
          went = __all_sync(0xffffffffu, wait_for(p, sh, &sh.empty[stage], (round - 1) & 1));
        if (!went) break;
        if (!skip) {
          if (lane == 0) {
            sh.bad[stage] = bad_pages;
            da::mbar_arrive_expect_tx(&sh.full[stage], __popc(pages) * rec);
          }
          __syncwarp();
          if (now >= 0) {
            uint8_t* to = ring + (size_t)stage * g_::STAGE + lane * rec;
            const uint8_t* from = p.pool + ((long long)now * p.Hkv + sg.kv) * p.page_bytes;
            if (bs <= kTok) {
              da::bulk_load(to, from, rec, &sh.full[stage]);
            } else {  // part of a page: codes and params of its rows from r on
              const int r = ((s.tile0 + i) * kTok) & (bs - 1);
              da::bulk_load(to, from + r * RB, eb * RB, &sh.full[stage]);
              da::bulk_load(to + eb * RB, from + (bs + r) * RB, eb * RB, &sh.full[stage]);
              const uint8_t* par = from + bs * D;
              da::bulk_load(to + eb * D, par + r * 4 * NG, eb * 4 * NG, &sh.full[stage]);
              da::bulk_load(to + eb * (D + 4 * NG), par + (bs + r) * 4 * NG, eb * 4 * NG,
                            &sh.full[stage]);
            }
          }
        }
        skip = false;
        if (++stage == p.stages) stage = 0, ++round;
      }
    }
    // After an abort: what was copied has to land before its memory is given back.
    if (!went || *(volatile int*)&sh.abort) {
      for (int i = 0; i < p.stages; ++i) {
        const int rounds = round + (i < stage ? 1 : 0);  // of this stage
        const bool unarmed = p.test_skip_arm && blockIdx.x == 0 && i == 0 && rounds == 1;
        if (rounds > 0 && !unarmed) da::mbar_wait(&sh.full[i], (rounds - 1) & 1, nullptr, p.wait_ns);
      }
    }
    __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- consumers
    da::setmaxnreg_inc<kConsumerRegs>();
    const int g = lane >> 2, c = lane & 3;
    // key of the 16 that row i of the MMA holds: tau(i) = i, tau(8 + i) = 8 + (i ^ 4).  Row j of V's
    // 16 x 16 bytes is key pi(j), which makes its bytes 4c .. 4c + 3 the keys of the MMA's k = 2c, 2c + 8, 2c + 1, 2c + 9.
    const int key_a = g, key_b = 8 + (g ^ 4);
    auto row_at = [&](int t) { return t * RB + (eb == 8 && t >= 8 ? rec - 8 * RB : 0); };
    auto par_at = [&](int t) { return t * 4 * NG + (eb == 8 && t >= 8 ? rec - 8 * 4 * NG : 0); };
    uint32_t k_lane, v_lane;  // byte offsets of this lane's rows from the 16 keys' first
    {
      const int j = lane & 7, t = lane & 8 ? 8 + (j ^ 4) : j;
      k_lane = row_at(t) + (((lane >> 4) ^ da::piece_xor<D>(t)) << 4);
      const int i = lane & 15, cc = i >> 2, w = i & 3;
      const int row = 2 * cc + (w >> 1);  // of tau's first half, or (odd w) of its second
      const int u = w & 1 ? 8 + (row ^ 4) : row;
      v_lane = row_at(u) + (((lane >> 4) ^ da::piece_xor<D>(u)) << 4);
    }
    const int par_a = par_at(key_a), par_b = par_at(key_b);
    const int rg = warp & (p.groups - 1), slot0 = warp / p.groups, slots = kWarps / p.groups;
    const uint32_t ring_u32 = da::smem_u32(ring);
    float* state = reinterpret_cast<float*>(scratch);
    uint4* qfrag = reinterpret_cast<uint4*>(scratch) + (size_t)rg * P * 2 * 32;
    int stage = 0, round = 0;
    Seg sg;
    while (next_seg(p, pre, walk, sg)) {
      Seq s;
      seq_info(p, sg.b, s);
      const int end = sg.i1 < 0 ? s.tiles : sg.i1;
      const int row0 = (sg.block * p.groups + rg) * kRows;  // first query row of the warp
      // ------------------------------------------------ Q: row g, dims 32 p + 8 c ..
      uint32_t qf[g_::QREG ? P * 2 : 1][4];  // hi of k = 2c.. and 2c + 8.., lo of the same
      float f[2], qs[NG][2];                 // factors and group sums of columns 2c, 2c + 1
      int lo[2], hi[2];
      {
        const int r = row0 + g;
        float x[P][8];
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (r < p.R) {
            const int t = r / p.G, h = sg.kv * p.G + (r - t * p.G);
            const float4* src = reinterpret_cast<const float4*>(
                p.q + (((long long)sg.b * p.T + t) * p.Hq + h) * D + 32 * i + 8 * c);
            const float4 a = src[0], b = src[1];
            x[i][0] = a.x, x[i][1] = a.y, x[i][2] = a.z, x[i][3] = a.w;
            x[i][4] = b.x, x[i][5] = b.y, x[i][6] = b.z, x[i][7] = b.w;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) most = max_nan(most, fabsf(x[i][j]));
        }
        most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const bool finite = most < INFINITY;
        // most < 2^e, e at least -100
        int e = (int)(__float_as_uint(most) >> 23) - 126;
        e = max(e, -100);
        const float up = finite ? __uint_as_float((uint32_t)(14 - e + 127) << 23) : 0.f;
        float back = __uint_as_float((uint32_t)(e - 14 + 127) << 23) * p.qscale;
        if (!finite) back = __uint_as_float(0x7fc00000u);
        float sum[NG] = {};
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[i][j] = finite ? x[i][j] * up : 0.f;
            sum[i / GP] += x[i][j];
          }
#pragma unroll
          for (int o = 0; o < 2; ++o) {  // low nibbles of a byte, high ones
            uint4 w;
            da::split_half2(x[i][o], x[i][o + 4], w.x, w.z);
            da::split_half2(x[i][o + 2], x[i][o + 6], w.y, w.w);
            if constexpr (g_::QREG) {
              qf[2 * i + o][0] = w.x, qf[2 * i + o][1] = w.y;
              qf[2 * i + o][2] = w.z, qf[2 * i + o][3] = w.w;
            } else {
              qfrag[(2 * i + o) * 32 + lane] = w;  // warps of the same rows write the same
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          sum[n] += __shfl_xor_sync(0xffffffffu, sum[n], 1);
          sum[n] += __shfl_xor_sync(0xffffffffu, sum[n], 2);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f[j] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + j));
#pragma unroll
          for (int n = 0; n < NG; ++n)
            qs[n][j] = __shfl_sync(0xffffffffu, sum[n], 4 * (2 * c + j)) * f[j];
          row_keys(p, s, (row0 + 2 * c + j) / p.G, lo[j], hi[j]);
        }
        __syncwarp();
      }
      // keys that every row sees
      int all_lo, all_hi, unused;
      row_keys(p, s, p.T - 1, all_lo, unused);
      row_keys(p, s, 0, unused, all_hi);

      float o[MT][4] = {}, acc[MT][4] = {};
      float zero_sum[NG][2] = {}, l[2] = {}, m[2] = {-INFINITY, -INFINITY};
      int chain = 0;
      for (int i = sg.i0; i < end; ++i) {
        wait_for(p, sh, &sh.full[stage], round & 1);
        const uint32_t bad = sh.bad[stage];
        const uint32_t base = ring_u32 + stage * g_::STAGE;
        for (int step = slot0; step < kTok / 16; step += slots) {
          const int tok = 16 * step, key0 = (s.tile0 + i) * kTok + tok;
          if (key0 >= s.hi || key0 + 16 <= s.lo) continue;
          const int piece = tok >> p.log2_eb, r0 = tok & (eb - 1);
          const uint32_t at = base + piece * rec;
          // -------------------------------------------- scores
          uint32_t kw[P][2];
#pragma unroll
          for (int i2 = 0; i2 < P / 2; ++i2)
            da::ldsm_x4((at + r0 * RB + k_lane) ^ (i2 << 5), kw[2 * i2][0], kw[2 * i2][1],
                        kw[2 * i2 + 1][0], kw[2 * i2 + 1][1]);
          const uint8_t* par = ring + (size_t)stage * g_::STAGE + piece * rec + eb * D + r0 * 4 * NG;
          uint32_t kp[2][NG], vp[2][NG];
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            kp[0][n] = *reinterpret_cast<const uint32_t*>(par + par_a + 4 * n);
            kp[1][n] = *reinterpret_cast<const uint32_t*>(par + par_b + 4 * n);
            vp[0][n] = *reinterpret_cast<const uint32_t*>(par + eb * 4 * NG + par_a + 4 * n);
            vp[1][n] = *reinterpret_cast<const uint32_t*>(par + eb * 4 * NG + par_b + 4 * n);
          }
          float x[4];  // keys a, a, b, b; columns 2c, 2c + 1
          {
            float u[4] = {}, z[4] = {};
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              float ah[4] = {}, al[4] = {};
#pragma unroll
              for (int i2 = n * GP; i2 < (n + 1) * GP; ++i2) {
                const uint32_t a0 = kw[i2][0], a1 = kw[i2][1], b0 = a0 >> 8, b1 = a1 >> 8;
#pragma unroll
                for (int o2 = 0; o2 < 2; ++o2) {
                  const uint32_t f0 = codes2(a0, o2), f1 = codes2(a1, o2);
                  const uint32_t f2 = codes2(b0, o2), f3 = codes2(b1, o2);
                  uint32_t q0, q1, q2, q3;
                  if constexpr (g_::QREG) {
                    q0 = qf[2 * i2 + o2][0], q1 = qf[2 * i2 + o2][1];
                    q2 = qf[2 * i2 + o2][2], q3 = qf[2 * i2 + o2][3];
                  } else {
                    const uint4 w = qfrag[(2 * i2 + o2) * 32 + lane];
                    q0 = w.x, q1 = w.y, q2 = w.z, q3 = w.w;
                  }
                  da::mma_f16_16816(ah, f0, f1, f2, f3, q0, q1);
                  da::mma_f16_16816(al, f0, f1, f2, f3, q2, q3);
                }
              }
              const float sa = half_lo(kp[0][n]) * 0x1p9f, sb = half_lo(kp[1][n]) * 0x1p9f;
              const float za = fmaf(sa, 0x1p-6f, half_hi(kp[0][n]));
              const float zb = fmaf(sb, 0x1p-6f, half_hi(kp[1][n]));
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                u[j] = fmaf(ah[j] + al[j], sa, u[j]);
                u[2 + j] = fmaf(ah[2 + j] + al[2 + j], sb, u[2 + j]);
                z[j] = fmaf(za, qs[n][j], z[j]);
                z[2 + j] = fmaf(zb, qs[n][j], z[2 + j]);
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = fmaf(u[j], f[j & 1], z[j]);
          }
          if (p.softcap2 > 0.f) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = soft_cap(x[j] * p.softcap_inv, p.softcap2);
          }
          // -------------------------------------------- masks
          const bool part = key0 < all_lo || key0 + 16 > all_hi || bad;
          uint32_t seen = 15u;
          if (part) {
            seen = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int t = j < 2 ? key_a : key_b, k = key0 + t;
              if (k >= lo[j & 1] && k < hi[j & 1] && !(bad >> ((tok + t) >> p.log2_eb) & 1))
                seen |= 1u << j;
              else
                x[j] = -INFINITY;
            }
          }
          // -------------------------------------------- reference and weights
          int ea = 0, eb2 = 0;  // largest value scale, as f16 bits
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            ea = max(ea, (int)(vp[0][n] & 0x7fffu));
            eb2 = max(eb2, (int)(vp[1][n] & 0x7fffu));
          }
          const float fa = (float)((ea >> 10) - 14), fb = (float)((eb2 >> 10) - 14);
          const bool out_of = x[0] + fa > m[0] + kSlack || x[1] + fa > m[1] + kSlack ||
                              x[2] + fb > m[0] + kSlack || x[3] + fb > m[1] + kSlack;
          if (__any_sync(0xffffffffu, out_of)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float n = fmaxf(x[j] + fa, x[2 + j] + fb);
#pragma unroll
              for (int off = 4; off < 32; off <<= 1)
                n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, off));
              n = fmaxf(n, m[j]);
              const float by = n == m[j] ? 1.f : da::ex2_ftz(m[j] - n);
              m[j] = n;
              l[j] *= by;
#pragma unroll
              for (int i2 = 0; i2 < NG; ++i2) zero_sum[i2][j] *= by;
#pragma unroll
              for (int i2 = 0; i2 < MT; ++i2) {
                o[i2][j] *= by, o[i2][2 + j] *= by;
                acc[i2][j] *= by, acc[i2][2 + j] *= by;
              }
            }
          }
          float w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[j] = da::ex2_ftz(x[j] + (kShift - m[j & 1]));
            if (part && !(seen >> j & 1)) w[j] = 0.f;
            l[j & 1] += w[j];
          }
          // -------------------------------------------- values
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const float sa = half_lo(vp[0][n]), sb = half_lo(vp[1][n]);
            const float za = fmaf(8.f, sa, half_hi(vp[0][n])), zb = fmaf(8.f, sb, half_hi(vp[1][n]));
            float ws[4] = {w[0] * sa, w[1] * sa, w[2] * sb, w[3] * sb};
            float wz[4] = {w[0] * za, w[1] * za, w[2] * zb, w[3] * zb};
            if (part) {  // a key that is not seen may have any scale and zero
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!(seen >> j & 1)) ws[j] = wz[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) zero_sum[n][j] += wz[j] + wz[2 + j];
            uint32_t h0, h1, l0, l1;
            da::split_half2(ws[0], ws[1], h0, l0);
            da::split_half2(ws[2], ws[3], h1, l1);
            h0 = da::movmatrix_trans(h0), h1 = da::movmatrix_trans(h1);
            l0 = da::movmatrix_trans(l0), l1 = da::movmatrix_trans(l1);
#pragma unroll
            for (int i2 = n * GP; i2 < (n + 1) * GP; ++i2) {
              // pieces come in pairs: lanes 16 to 31 address the odd one
              uint32_t r0_, r1_, r2_, r3_;
              da::ldsm_b8_x2_trans((at + (eb + r0) * RB + v_lane) ^ (i2 / 2 << 5), r0_, r1_, r2_, r3_);
              const uint32_t a0 = i2 & 1 ? r2_ : r0_, a1 = i2 & 1 ? r3_ : r1_;
              const uint32_t b0 = a0 >> 8, b1 = a1 >> 8;
#pragma unroll
              for (int o2 = 0; o2 < 2; ++o2) {
                const uint32_t f0 = codes2(a0, o2), f1 = codes2(a1, o2);
                const uint32_t f2 = codes2(b0, o2), f3 = codes2(b1, o2);
                da::mma_f16_16816(acc[2 * i2 + o2], f0, f1, f2, f3, h0, h1);
                da::mma_f16_16816(acc[2 * i2 + o2], f0, f1, f2, f3, l0, l1);
              }
            }
          }
          if (++chain == kChain) {
            chain = 0;
#pragma unroll
            for (int i2 = 0; i2 < MT; ++i2)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[i2][j] += acc[i2][j], acc[i2][j] = 0.f;
          }
        }
        __syncwarp();
        if (lane == 0) da::mbar_arrive(&sh.empty[stage]);
        if (++stage == p.stages) stage = 0, ++round;
      }
      // ------------------------------------------------ the warps' states to one
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l[j] += __shfl_xor_sync(0xffffffffu, l[j], off);
#pragma unroll
          for (int n = 0; n < NG; ++n)
            zero_sum[n][j] += __shfl_xor_sync(0xffffffffu, zero_sum[n][j], off);
        }
      }
      if (!g_::QREG) da::named_bar_sync(1, 32 * kWarps);  // Q's fragments are read
      if (g == 0) {
        sh.ml[warp][2 * c] = make_float2(m[0], l[0]);
        sh.ml[warp][2 * c + 1] = make_float2(m[1], l[1]);
      }
#pragma unroll
      for (int i2 = 0; i2 < P; ++i2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // row of V: 32 i2 + 2 g (+ 16): low nibble and high one side by side
          const float z = zero_sum[i2 / GP][j & 1];
          float2 v;
          v.x = fmaf(o[2 * i2][j] + acc[2 * i2][j], 0x1p9f, z);
          v.y = fmaf(o[2 * i2 + 1][j] + acc[2 * i2 + 1][j], 0x1p9f, z);
          *reinterpret_cast<float2*>(state + (warp * kRows + 2 * c + (j & 1)) * g_::COL + 32 * i2 +
                                     2 * g + (j & 2 ? 16 : 0)) = v;
        }
      }
      da::named_bar_sync(1, 32 * kWarps);
      for (int i = tid; i < p.groups * kRows * (D / 4); i += 32 * kWarps) {
        const int row = i / (D / 4), d = i % (D / 4) * 4, grp = row / kRows, col = row % kRows;
        const int r = sg.block * p.groups * kRows + row;
        if (r >= p.R) continue;
        float top = -INFINITY;
        for (int w = grp; w < kWarps; w += p.groups) top = fmaxf(top, sh.ml[w][col].x);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float tl = 0.f;
        for (int w = grp; w < kWarps; w += p.groups) {
          const float2 ml = sh.ml[w][col];
          const float by = ml.x == top ? 1.f : da::ex2_ftz(ml.x - top);
          const float4 v = *reinterpret_cast<const float4*>(state + (w * kRows + col) * g_::COL + d);
          sum.x = fmaf(by, v.x, sum.x), sum.y = fmaf(by, v.y, sum.y);
          sum.z = fmaf(by, v.z, sum.z), sum.w = fmaf(by, v.w, sum.w);
          tl = fmaf(by, ml.y, tl);
        }
        if (sg.slot < 0) {
          const int t = r / p.G, h = sg.kv * p.G + (r - t * p.G);
          const long long to = ((long long)sg.b * p.T + t) * p.Hq + h;
          const float inv = tl == 0.f ? 0.f : 1.f / tl;
          *reinterpret_cast<float4*>(p.out + to * D + d) =
              make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
          if (d == 0 && p.lse)
            p.lse[to] = tl == 0.f ? -INFINITY : (top - kShift + log2f(tl)) * kLn2;
        } else {
          const long long to = (long long)(blockIdx.x * 2 + sg.slot) * p.groups * kRows + row;
          *reinterpret_cast<float4*>(p.part_o + to * D + d) = sum;
          if (d == 0) p.part_ml[to] = make_float2(top, tl);
        }
      }
      da::named_bar_sync(1, 32 * kWarps);  // the states are read
    }
    if (p.split) {
      // the unit that is cut at this CTA's end, if it starts here: who has its parts
      if (tid == 0) {
        int4 d = make_int4(-1, 0, 0, 0);
        if (walk.n > 0 && sg.slot >= 0 && sg.i0 == 0) {
          const int nt = pre[sg.b + 1] - pre[sg.b];
          const int last = pre[sg.b] * walk.upb + (sg.kv * p.blocks + sg.block + 1) * nt - 1;
          // the CTA whose share holds tile `last`
          int cta = (int)(((long long)last * shares) / total);
          while (cta + 1 < shares && share_start(cta + 1, total, shares) <= last) ++cta;
          d = make_int4(sg.b, sg.kv * p.blocks + sg.block, sg.slot, cta);
        }
        p.desc[blockIdx.x] = d;
      }
      // sequences without a key to see
      for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (pre[b + 1] != pre[b]) continue;
        const long long rows = (long long)p.T * p.Hq;
        float4* to = reinterpret_cast<float4*>(p.out + b * rows * D);
        for (long long i = tid; i < rows * (D / 4); i += 32 * kWarps)
          to[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.lse)
          for (long long i = tid; i < rows; i += 32 * kWarps) p.lse[b * rows + i] = -INFINITY;
      }
    }
  }
  __syncthreads();
  if (tid == 0 && sh.abort && p.dev_status) atomicOr(p.dev_status, DA_DEV_TIMEOUT);
}

// Adds up the states of a unit that CTAs share: block (i, y) rows 2y, 2y + 1 of the unit that starts in CTA
// i's share and is cut at its end.
constexpr int kMergeThreads = 128, kMergeRows = 2, kMaxParts = 1024;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) q4_merge_kernel(const __grid_constant__ Q4Params p) {
  __shared__ float by[kMergeRows][kMaxParts];
  __shared__ float2 ml[kMergeRows];
  da::wait_for_grid_before();
  da::let_next_grid_start();
  const int4 d = p.desc[blockIdx.x];
  if (d.x < 0) return;
  const int rows = p.groups * kRows, parts = d.w - blockIdx.x + 1;
  const int kv = d.y / p.blocks, block = d.y - kv * p.blocks;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // place of part i of row r: the first one is in the slot that d names, the others in slot 0
  auto place = [&](int i, int r) {
    return (long long)((blockIdx.x + i) * 2 + (i ? 0 : d.z)) * rows + blockIdx.y * kMergeRows + r;
  };
  if (warp < kMergeRows) {
    float top = -INFINITY, l = 0.f;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.part_ml[place(i, warp)].x);
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    for (int i = lane; i < parts; i += 32) {
      const float2 x = p.part_ml[place(i, warp)];
      const float f = x.x == top ? 1.f : da::ex2_ftz(x.x - top);
      by[warp][i] = f;
      l = fmaf(f, x.y, l);
    }
    for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane == 0) ml[warp] = make_float2(top, l);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kMergeRows * D / 4; i += kMergeThreads) {
    const int r = i / (D / 4), col = i % (D / 4) * 4;
    const int row = block * rows + blockIdx.y * kMergeRows + r;
    if (row >= p.R) continue;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + place(k, r) * D + col);
      const float f = by[r][k];
      sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y);
      sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
    }
    const float l = ml[r].y, inv = l == 0.f ? 0.f : 1.f / l;
    const int t = row / p.G, h = kv * p.G + (row - t * p.G);
    const long long to = ((long long)d.x * p.T + t) * p.Hq + h;
    *reinterpret_cast<float4*>(p.out + to * D + col) =
        make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
    if (col == 0 && p.lse)
      p.lse[to] = l == 0.f ? -INFINITY : (ml[r].x - kShift + log2f(l)) * kLn2;
  }
}

// ------------------------------------------------------------------ host
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Shape {
  int groups, blocks, chunk;  // row groups of a unit, units of a kv head, sequences of a launch
};

int check(const da_params* p, int group, int q_len, Shape& s) {
  int st = da::check_paged(p);
  if (st == DA_OK) st = da::check_q4(p, group);
  if (st != DA_OK) return st;
  if (q_len < 1) return DA_ERR_INVALID;
  const long long cap = (long long)p->max_blocks_per_seq * p->block_size;
  const long long rows = (long long)q_len * (p->num_q_heads / p->num_kv_heads);
  if (cap > 0x7fffffffLL - 1024 || rows > 0x7fffffffLL - 1024) return DA_ERR_UNSUPPORTED;
  const long long groups = (rows + kRows - 1) / kRows;
  s.groups = 1;
  while (s.groups < groups && s.groups < kMaxGroups) s.groups *= 2;
  const long long blocks = (groups + s.groups - 1) / s.groups;
  // tiles of a launch count in 31 bits
  const long long tiles = (cap / kTok + 2) * p->num_kv_heads * blocks;
  const long long most = (0x7fffffffLL - 1024) / tiles;
  if (most < 1) return DA_ERR_UNSUPPORTED;
  s.blocks = (int)blocks;
  s.chunk = (int)(most < kMaxBatch ? most : kMaxBatch);
  return DA_OK;
}

struct Layout {
  size_t desc, ml, o, total;
};
Layout layout(int sms, int groups, int D) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Layout w;
  const size_t rows = (size_t)sms * 2 * groups * kRows;
  w.desc = 0;
  w.ml = up(sizeof(int4) * sms);
  w.o = w.ml + up(rows * sizeof(float2));
  w.total = w.o + up(rows * D * sizeof(float));
  return w;
}

template <int D, int NG>
cudaError_t launch(Q4Params& k, int grid, cudaStream_t s) {
  using g_ = Geo<D, NG>;
  constexpr int kMost = 227 * 1024 - 2048;  // dynamic shared memory, Shared beside it
  const int pre = k.split ? (k.B + 1) * 4 : 0;
  int stages = (kMost - g_::UNION - pre) / g_::STAGE;
  if (stages > 16) stages = 16;
  k.stages = stages;
  const int smem = stages * g_::STAGE + g_::UNION + pre;
  cudaError_t err = cudaFuncSetAttribute(q4_kernel<D, NG>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (err != cudaSuccess) return err;
  err = da::launch_early(q4_kernel<D, NG>, grid, kThreads, smem, s, k);
  if (err != cudaSuccess || !k.split) return err;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, k.groups * kRows / kMergeRows);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_merge_kernel<D>, k);
}

cudaError_t launch(Q4Params& k, int D, int group, int grid, cudaStream_t s) {
  switch (D * 1000 + group) {
    case 64032: return launch<64, 2>(k, grid, s);
    case 64064: return launch<64, 1>(k, grid, s);
    case 128032: return launch<128, 4>(k, grid, s);
    case 128064: return launch<128, 2>(k, grid, s);
    case 128128: return launch<128, 1>(k, grid, s);
    case 256032: return launch<256, 8>(k, grid, s);
    case 256064: return launch<256, 4>(k, grid, s);
    default: return launch<256, 2>(k, grid, s);
  }
}

// A call's kernels hand over through its workspace: they are enqueued without another's between them.
std::mutex& workspace_mutex(const void* workspace) {
  static std::mutex locks[64];
  return locks[(reinterpret_cast<uintptr_t>(workspace) >> 8) % 64];
}

}  // namespace

extern "C" {

size_t decode_attn_paged_q4_workspace_size(const da_params* p, int32_t q_len) {
  Shape s;
  int sms = 0;
  if (check(p, da::kQ4MinGroup, q_len, s) != DA_OK || da::device_sms(&sms) != DA_OK) return 0;
  return layout(sms, s.groups, p->head_dim).total;
}

int decode_attn_paged_q4(const da_params* p, int32_t group, int32_t q_len, const float* q,
                         const uint8_t* pool, const int32_t* block_table,
                         const int32_t* seq_lens, const int32_t* q_pos, float* out, float* lse,
                         void* workspace, size_t workspace_bytes, int32_t* dev_status,
                         void* stream) {
  Shape shape;
  int st = check(p, group, q_len, shape);
  if (st != DA_OK) return st;
  if (!q || !pool || !block_table || !seq_lens || !out) return DA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || (q_pos && !aligned(q_pos, 4)) || (lse && !aligned(lse, 4)) ||
      (dev_status && !aligned(dev_status, 4)) || !aligned(workspace, 256))
    return DA_ERR_INVALID;
  if (!workspace && workspace_bytes) return DA_ERR_INVALID;
  // rows of out are written while others' q is still to be read
  const long long values = (long long)p->batch * q_len * p->num_q_heads * p->head_dim;
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
  if ((qa < oa ? oa - qa : qa - oa) < (unsigned long long)values * 4) return DA_ERR_INVALID;
  if (p->batch == 0) return DA_OK;
  int sms = 0;
  st = da::device_sms(&sms);
  if (st != DA_OK) return st;
  const Layout w = layout(sms, shape.groups, p->head_dim);
  if (workspace && workspace_bytes < w.total) return DA_ERR_WORKSPACE;
  if (sms > kMaxParts) return DA_ERR_UNSUPPORTED;
  Q4Params k = {};
  k.pool = pool;
  k.dev_status = dev_status;
  k.T = q_len;
  k.G = p->num_q_heads / p->num_kv_heads;
  k.R = k.T * k.G;
  k.Hq = p->num_q_heads;
  k.Hkv = p->num_kv_heads;
  while ((1 << k.log2_bs) < p->block_size) ++k.log2_bs;
  const int eb = p->block_size < kTok ? p->block_size : kTok;
  while ((1 << k.log2_eb) < eb) ++k.log2_eb;
  k.max_blocks = p->max_blocks_per_seq;
  k.num_blocks = p->num_blocks;
  k.window = p->sliding_window;
  k.causal = p->causal;
  k.groups = shape.groups;
  k.blocks = shape.blocks;
  k.qscale = da::base2_scale(p);
  k.softcap2 = p->softcap > 0.f ? p->softcap * 1.4426950408889634f : 0.f;
  k.softcap_inv = k.softcap2 > 0.f ? (float)(1.0 / (double)k.softcap2) : 0.f;
  k.page_bytes = da::q4_page_bytes(p->block_size, p->head_dim, group);
  k.wait_ns = da::wait_limit();
  k.test_skip_arm = da::skip_first_arm();
  if (workspace) {
    char* ws = static_cast<char*>(workspace);
    k.desc = reinterpret_cast<int4*>(ws + w.desc);
    k.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    k.part_o = reinterpret_cast<float*>(ws + w.o);
  }
  const long long row = (long long)q_len * p->num_q_heads;
  const std::lock_guard<std::mutex> unbroken(workspace_mutex(workspace));
  for (int b0 = 0; b0 < p->batch; b0 += shape.chunk) {
    k.B = p->batch - b0 < shape.chunk ? p->batch - b0 : shape.chunk;
    k.q = q + b0 * row * p->head_dim;
    k.out = out + b0 * row * p->head_dim;
    k.lse = lse ? lse + b0 * row : nullptr;
    k.table = block_table + (long long)b0 * k.max_blocks;
    k.seq_lens = seq_lens + b0;
    k.q_pos = q_pos ? q_pos + b0 : nullptr;
    k.units = k.B * k.Hkv * k.blocks;
    // Short sequences run whole: a cut unit costs a second kernel.
    k.split = workspace && !(p->max_seq_len > 0 && p->max_seq_len <= 512 && k.units <= 2 * sms);
    const int grid = k.split || k.units > sms ? sms : k.units;
    if (launch(k, p->head_dim, group, grid, static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return DA_ERR_CUDA;
  }
  return DA_OK;
}

}  // extern "C"
