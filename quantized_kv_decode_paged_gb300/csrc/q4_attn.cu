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
// f16's smallest step at m.  mma.sync adds with truncation, so a sum takes chain_keys keys at most and is
// then added up in f32.
//
// Work.  A unit is (sequence, kv head, up to 64 query rows: query tokens x heads of the kv head), a tile 16
// to 64 of its keys (4.25 to 5 KB of codes, scales and zeros).  The tiles of all units stand in one row that is cut
// into equal shares, one a warp (or one for the two or four warps that take a unit's rows, 8 or 16 each): a
// warp copies its tiles into a ring of its own, 16 bytes a lane at a time (codes and scales of keys and values
// lie side by side in a page of a head), waits for them and works them off, and nothing of it waits for another
// warp.  32 keys (D = 256: 16) x 8 rows at a time: S^T = K Q^T and O^T += V^T P^T with mma.m16n8k16, keys
// and value columns as M, so that 8 rows of Q fill N.  A unit that ends in another share than it began in
// leaves its parts' states in the workspace; q4_merge_kernel adds them up.  The row order of the 16 keys (tau
// below) is such that the fragments of K by ldmatrix and of V by its transposing byte form meet in one layout and
// no bank twice.
//
// Measured (one GB300): 128 sequences of 2048 to 24,000 keys, 8 kv heads, 64 query heads, D = 128: 334 us for
// 1.26 GB, 56% of the copy bandwidth.  The copies alone take 215 us, everything but the copies 272, of which 119 are
// left without the matrix products: these and what makes their operands add up, the copies
// hide for the most part.  Splitting by CTA with a common ring and producer warps took 515 us, by warp with
// bulk copies 381 us.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "../../include/decode_attn.h"
#include "launch.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace {

constexpr int kRows = 8;                // query rows of a group: N of a product
constexpr int kMaxWarps = 4;            // warps of a unit
constexpr int kMaxBatch = 1024;         // sequences of a launch
// Keys of a warp between f32 additions.  With 8 rows a product, whose sums take both terms, 128 sequences of 2048
// to 24,000 keys: 326 us and an error of 2.6e-6 with 256, 328 and 1.7e-6 with 128, 334 and 1.3e-6 with 64, which
// is f32's own, 345 and 1.3e-6 with 32.  With 4 rows and a sum a term, 24 sequences of 20,000 to 40,000 keys: 172
// us and 7.7e-7 with 256, 177 and 9e-7 with 64.
constexpr int chain_keys(bool pack) { return pack ? 256 : 64; }
constexpr float kShift = 10.f, kSlack = 5.f;
constexpr float kLn2 = 0.6931471805599453f;
// The reference of a row before its first key of weight: finite, so that scores of -inf (below f32's range) that
// come before it weigh 0 and not 2^(-inf + inf).
constexpr float kLeast = -3.402823466e38f;

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
  int warps, blocks;   // warps of a unit (a power of two), units of a kv head
  int unit_rows;       // query rows of a unit
  int log2_eb;         // rows of a page's piece in a tile, min(block size, tile)
  int shares;          // of the launch
  float qscale, softcap2, softcap_inv;
  long long page_bytes;
  uint32_t stride;     // bytes from a page to the next: below 2^32
  // workspace
  int* pre;         // [B + 1] tiles of the sequences before each
  float2* part_ml;  // [shares][2][unit_rows]: reference and sum
  float* part_o;    // [shares][2][unit_rows][D]
};

// ------------------------------------------------------------------ what a sequence sees
struct Seq {
  int len, lo, hi;  // keys [lo, hi) are seen by some row
  int qp;           // position of query token 0
  int tile0, tiles;
};

template <int TOK>
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
  s.qp = (int)qp;
  s.tile0 = (int)(lo / TOK);
  s.tiles = hi > lo ? (int)((hi + TOK - 1) / TOK) - s.tile0 : 0;
  return flags;
}

// Keys [lo, hi) that query token t sees.
__device__ __forceinline__ void row_keys(const Q4Params& p, const Seq& s, int t, int& lo, int& hi) {
  const long long qp = (long long)s.qp + t;
  const long long first = p.window > 0 && qp >= p.window ? qp - p.window + 1 : 0;
  lo = (int)(first < 0x7fffffff ? first : 0x7fffffff);  // past every key
  hi = p.causal && qp + 1 < s.len ? (int)(qp + 1) : s.len;
  if (s.tiles == 0) hi = lo;
}

// ------------------------------------------------------------------ shares
// Of `total` tiles share i has [start(i), start(i + 1)); with fewer tiles than shares the last ones have none.
struct Shares {
  int total, n;
  __device__ __forceinline__ Shares(int tiles, int shares)
      : total(tiles), n(tiles < shares ? tiles : shares) {}
  // x * y / z, in 32 bits where the products of this launch fit into them (64 sequences behind a window of 4096: 147
  // us, else 155)
  __device__ __forceinline__ int ratio(int x, int y, int z) const {
    if ((long long)total * n <= 0xffffffffLL) return (int)((uint32_t)x * (uint32_t)y / (uint32_t)z);
    return (int)((long long)x * y / z);
  }
  __device__ __forceinline__ int start(int i) const { return ratio(i, total, n); }
  __device__ __forceinline__ int of(int tile) const {  // whose it is
    int i = ratio(tile, n, total);
    while (i + 1 < n && start(i + 1) <= tile) ++i;
    return i;
  }
};

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

// As mma_f16_16816, free to move among what surrounds it.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first of a sum.
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 16 bytes to shared memory, past L1, with the next ones' line to L2.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// NG params of a row side by side in shared memory.
template <int NG>
__device__ __forceinline__ void load_params(uint32_t at, uint32_t (&w)[NG]) {
  if constexpr (NG == 1) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
  } else if constexpr (NG == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < NG / 4; ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(at + 16 * i)
                   : "memory");
  }
}

// ROWS: query rows of a warp, 4, 8 or 16.
template <int D, int NG, int ROWS>
struct Geo {
  static constexpr int RG = ROWS == 16 ? 2 : 1;  // groups of kRows rows
  static constexpr bool BIG = D == 256 || (D == 128 && RG == 2);  // sums fill the registers
  static constexpr int P = D / 32;         // 16-byte pieces of a row
  static constexpr int GP = P / NG;        // pieces of a group
  static constexpr int RB = D / 2;         // bytes of a row's codes
  static constexpr int ROW = D + 8 * NG;   // bytes of a key's and a value's row
  static constexpr int TOK = 4096 / D;     // keys of a tile
  static constexpr int LOG2_TOK = D == 64 ? 6 : D == 128 ? 5 : 4;
  static constexpr int H = BIG ? 1 : 2;    // MMA tiles of 16 keys that are worked off together
  static constexpr int STAGE = TOK * ROW;  // codes of keys, of values, params of keys, of values
  static constexpr int CODES = TOK * RB;
  static constexpr int WARPS = BIG ? 8 : 12;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr bool QREG = !BIG;       // Q's fragments in registers, else in shared memory
  static constexpr int STATE = RG * kRows * D * 4;  // sums of a warp in shared memory
  static constexpr int QBYTES = QREG ? 0 : RG * P * 2 * 512;
  static constexpr int kMost = 227 * 1024 - 2048;  // dynamic shared memory, Shared beside it
  static constexpr int FIT = (kMost - (kMaxBatch + 1) * 4) / WARPS - STATE - QBYTES;
  static constexpr int STAGES = FIT / STAGE < 4 ? FIT / STAGE : 4;  // of a warp's ring
  static constexpr int SMEM = WARPS * (STAGES * STAGE + STATE + QBYTES);
  static_assert(STAGES >= 2, "a warp's ring has two stages at least");
};

template <int WARPS, int STAGES>
struct Shared {
  uint32_t bad[WARPS][STAGES];  // pages of a tile that are outside the pool
  int warp_sum[WARPS];
};

// ROWS 4 (PACK): at most four query rows a unit, whose two terms share one MMA operand: rows 0 to 3 of N are the first
// terms, 4 to 7 the second ones, so that half the MMAs do.  ROWS 16: two groups of
// rows share the operands that are made of the codes.
template <int D, int NG, int ROWS>
__global__ void __launch_bounds__(Geo<D, NG, ROWS>::THREADS, 1)
    q4_kernel(const __grid_constant__ Q4Params p) {
  using g_ = Geo<D, NG, ROWS>;
  constexpr bool PACK = ROWS == 4;
  constexpr int RG = g_::RG, WROWS = RG * kRows;  // rows of a warp, of which PACK uses four
  constexpr int P = g_::P, GP = g_::GP, RB = g_::RB, MT = 2 * P, H = g_::H, TOK = g_::TOK;
  constexpr int STAGES = g_::STAGES;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Shared<g_::WARPS, STAGES> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = da::smem_u32(dyn) + warp * (STAGES * g_::STAGE);
  float* state = reinterpret_cast<float*>(dyn + g_::WARPS * STAGES * g_::STAGE + warp * g_::STATE);
  uint4* qfrag = reinterpret_cast<uint4*>(
      dyn + g_::WARPS * (STAGES * g_::STAGE + g_::STATE) + warp * g_::QBYTES);
  int* pre = reinterpret_cast<int*>(dyn + g_::SMEM);
  const int eb = 1 << p.log2_eb, bs = 1 << p.log2_bs;
  const int upb = p.Hkv * p.blocks;  // units of a sequence

  da::wait_for_grid_before();
  da::let_next_grid_start();

  // ------------------------------------------------ tiles of the sequences before each
  int total = 0;
  {
    const int per = (p.B + g_::THREADS - 1) / g_::THREADS, b0 = min(tid * per, p.B);
    const int b1 = min(b0 + per, p.B);
    int mine = 0, bad = 0;
    for (int b = b0; b < b1; ++b) {
      Seq s;
      bad |= seq_info<TOK>(p, b, s);
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
    for (int i = 0; i < g_::WARPS; ++i) {
      if (i < warp) run += sh.warp_sum[i];
      total += sh.warp_sum[i];
    }
    for (int b = b0; b < b1; ++b) {
      run += pre[b + 1];
      pre[b + 1] = run;
      if (blockIdx.x == 0) p.pre[b + 1] = run;
    }
    if (tid == 0) {
      pre[0] = 0;
      if (blockIdx.x == 0) p.pre[0] = 0;
    }
    __syncthreads();
  }
  // From here on a warp is by itself.  Its row group of the units, its share of the tiles.
  const int slots = g_::WARPS / p.warps, rg = warp / slots;
  const int share = blockIdx.x * slots + (warp - rg * slots);
  const Shares shares(total * upb, p.shares);
  if (share >= shares.n) return;
  int tile = shares.start(share), segs = 0;
  const int tile_end = shares.start(share + 1);
  int seq = 0;  // the sequence that holds the first tile
  for (int hi = p.B; hi - seq > 1;) {
    const int mid = (seq + hi) / 2;
    if ((long long)pre[mid] * upb <= tile) seq = mid;
    else hi = mid;
  }

  // A unit's part.
  struct Part {
    Seq s;
    int b, kv, block;
    int i0, n;  // its first tile, of the sequence's; tiles
    int slot;   // -1: the whole unit; else the place of its state among the share's
    const uint8_t* base;  // this lane's 16 bytes of page 0 of the kv head
  };
  auto next_part = [&](Part& a) {
    if (tile >= tile_end) return false;
    while ((long long)pre[seq + 1] * upb <= tile) ++seq;
    const int nt = pre[seq + 1] - pre[seq], rel = tile - pre[seq] * upb, unit = rel / nt;
    a.b = seq;
    a.kv = unit / p.blocks;
    a.block = unit - a.kv * p.blocks;
    a.i0 = rel - unit * nt;
    a.n = min(nt - a.i0, tile_end - tile);
    a.slot = a.n == nt ? -1 : segs ? 1 : 0;
    a.base = p.pool + a.kv * p.page_bytes + 16 * lane;
    seq_info<TOK>(p, seq, a.s);
    tile += a.n;
    ++segs;
    return true;
  };

  // ------------------------------------------------ copies
  // Block ids are loaded 32 at a time, lane by lane: piece lane % pieces of tile lane / pieces of a batch of
  // tiles, a batch ahead of the copies.
  const int log2_pieces = g_::LOG2_TOK - p.log2_eb;
  const int batch = 32 >> log2_pieces, my_tile = lane >> log2_pieces;
  const int my_piece = lane & ((1 << log2_pieces) - 1);
  int id = -1, id_next = -1;  // of this lane's piece in this batch and the next; -1: not read, -2: outside
  uint32_t bad_pages = 0;     // of this batch: lanes with a piece outside the pool
  auto block_id = [&](const Part& a, int n) {
    const int k = (a.s.tile0 + a.i0 + n) * TOK + (my_piece << p.log2_eb);
    if (n >= a.n || k >= a.s.hi || k + eb <= a.s.lo) return -1;
    const int x = p.table[(long long)a.b * p.max_blocks + (k >> p.log2_bs)];
    return x >= 0 && x < p.num_blocks ? x : -2;
  };
  int put = 0, got = 0;  // stage of the next copy, of the next tile to work off
  // Tile n of the part, and a group of copies to wait for in any case.  (Bulk copies with barriers, which lanes
  // issue for themselves one by one, took 1100 cycles a tile of a warp's time.)
  auto copy = [&](const Part& a, int n) {
    if (n < a.n) {
      const int j = n & (batch - 1);
      if (j == 0) {
        id = id_next;
        id_next = block_id(a, n + batch + my_tile);
        bad_pages = __ballot_sync(0xffffffffu, id == -2);
        if (bad_pages && lane == 0 && p.dev_status) atomicOr(p.dev_status, DA_DEV_BAD_BLOCK);
      }
      const uint32_t those = (2u << ((1 << log2_pieces) - 1)) - 1;  // pieces of a tile
      if (lane == 0) sh.bad[warp][put] = bad_pages >> (j << log2_pieces) & those;
      const uint32_t to = ring + put * g_::STAGE + 16 * lane;
      auto pieces = [&](auto rows) {  // of `rows` keys each
        constexpr int EB = decltype(rows)::value, PAR = EB * 4 * NG;  // keys' params, values' params
#pragma unroll
        for (int i = 0; i < TOK / EB; ++i) {
          const int x = __shfl_sync(0xffffffffu, id, j * (TOK / EB) + i);
          if (x < 0) continue;
          const uint8_t* k = a.base + (unsigned long long)(uint32_t)x * p.stride;
          if (EB == TOK && bs > TOK)  // a part of a page: from this row on
            k += (((a.s.tile0 + a.i0 + n) * TOK) & (bs - 1)) * RB;
          const uint8_t* v = k + bs * RB;
          const uint32_t dst = to + i * EB * RB;
#pragma unroll
          for (int at = 0; at < EB * RB; at += 512)
            if (EB * RB >= 512 || 16 * lane < EB * RB) {
              copy16(dst + at, k + at);
              copy16(dst + g_::CODES + at, v + at);
            }
          const uint8_t* par = k + bs * D - 16 * lane;  // of the piece's keys
          if (EB == TOK && bs > TOK) par -= (((a.s.tile0 + a.i0 + n) * TOK) & (bs - 1)) * (RB - 4 * NG);
          const uint32_t pdst = to - 16 * lane + 2 * g_::CODES + i * PAR;
          if constexpr (PAR <= 256) {  // both in one go
            const int v2 = lane / (PAR / 16), off = lane % (PAR / 16) * 16;
            if (lane < PAR / 8) copy16(pdst + v2 * TOK * 4 * NG + off, par + v2 * bs * 4 * NG + off);
          } else if (16 * lane < PAR) {
            copy16(pdst + 16 * lane, par + 16 * lane);
            copy16(pdst + TOK * 4 * NG + 16 * lane, par + bs * 4 * NG + 16 * lane);
          }
        }
      };
      if (eb == TOK) pieces(std::integral_constant<int, TOK>());
      else if (eb == 8) pieces(std::integral_constant<int, 8>());
      else if (eb == 16) pieces(std::integral_constant<int, 16>());
      else if constexpr (TOK == 64) pieces(std::integral_constant<int, 32>());
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++put == STAGES) put = 0;
  };

  const int g = lane >> 2, c = lane & 3;
  const int col = PACK ? 2 * (c & 1) : 2 * c;  // query row of the lane's first column, of kRows
  // key of the 16 that row i of the MMA holds: tau(i) = i, tau(8 + i) = 8 + (i ^ 4).  Row j of V's
  // 16 x 16 bytes is key pi(j), which makes its bytes 4c .. 4c + 3 the keys of the MMA's k = 2c, 2c + 8,
  // 2c + 1, 2c + 9.
  const int key_a = g, key_b = 8 + (g ^ 4);
  uint32_t k_lane, v_lane;  // byte offsets of this lane's rows from the 16 keys' first
  {
    const int j = lane & 7, t = lane & 8 ? 8 + (j ^ 4) : j;
    k_lane = t * RB + (((lane >> 4) ^ da::piece_xor<D>(t)) << 4);
    const int i = lane & 15, cc = i >> 2, w = i & 3;
    const int row = 2 * cc + (w >> 1);  // of tau's first half, or (odd w) of its second
    const int u = w & 1 ? 8 + (row ^ 4) : row;
    v_lane = g_::CODES + u * RB + (((lane >> 4) ^ da::piece_xor<D>(u)) << 4);
  }
  // a lane's sums, accumulator i
  auto state_at = [&](int i) { return reinterpret_cast<float4*>(state) + 32 * i + lane; };

  Part a;
  while (next_part(a)) {
    const int row0 = (a.block * p.warps + rg) * WROWS;  // first query row of the warp
    // ------------------------------------------------ Q: row g of a group, dims 32 p + 8 c ..
    float x[RG][P][8];
#pragma unroll
    for (int gr = 0; gr < RG; ++gr) {
      const int r = row0 + kRows * gr + (PACK ? g & 3 : g);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float (&y)[8] = x[gr][i];
        if (r < p.R) {
          const int t = r / p.G, h = a.kv * p.G + (r - t * p.G);
          const float4* src = reinterpret_cast<const float4*>(
              p.q + (((long long)a.b * p.T + t) * p.Hq + h) * D + 32 * i + 8 * c);
          const float4 y0 = src[0], y1 = src[1];
          y[0] = y0.x, y[1] = y0.y, y[2] = y0.z, y[3] = y0.w;
          y[4] = y1.x, y[5] = y1.y, y[6] = y1.z, y[7] = y1.w;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = 0.f;
        }
      }
    }
    id_next = block_id(a, my_tile);
#pragma unroll 1
    for (int n = 0; n < STAGES; ++n) copy(a, n);
    constexpr int QW = PACK ? 2 : 4;  // words of a fragment: k = 2c.. and 2c + 8.. of the first term, the second
    uint32_t qf[g_::QREG ? RG * P * 2 : 1][QW];
    float2 f[RG], qs[RG][NG];  // factors and group sums of the lane's columns
    int lo[RG][2], hi[RG][2];
#pragma unroll
    for (int gr = 0; gr < RG; ++gr) {
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) most = max_nan(most, fabsf(x[gr][i][j]));
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
        float (&y)[8] = x[gr][i];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[j] = finite ? y[j] * up : 0.f;
          sum[i / GP] += y[j];
        }
#pragma unroll
        for (int o = 0; o < 2; ++o) {  // low nibbles of a byte, high ones
          uint4 w;
          da::split_half2(y[o], y[o + 4], w.x, w.z);
          da::split_half2(y[o + 2], y[o + 6], w.y, w.w);
          if (PACK && g >= 4) w.x = w.z, w.y = w.w;
          const int at = gr * P * 2 + 2 * i + o;
          if constexpr (g_::QREG) {
            qf[at][0] = w.x, qf[at][1] = w.y;
            if constexpr (!PACK) qf[at][2] = w.z, qf[at][3] = w.w;
          } else if constexpr (PACK) {
            reinterpret_cast<uint2*>(qfrag)[at * 32 + lane] = make_uint2(w.x, w.y);
          } else {
            qfrag[at * 32 + lane] = w;  // read back by this lane alone
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        sum[n] += __shfl_xor_sync(0xffffffffu, sum[n], 1);
        sum[n] += __shfl_xor_sync(0xffffffffu, sum[n], 2);
      }
      f[gr].x = __shfl_sync(0xffffffffu, back, 4 * col);
      f[gr].y = __shfl_sync(0xffffffffu, back, 4 * col + 4);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        qs[gr][n].x = __shfl_sync(0xffffffffu, sum[n], 4 * col) * f[gr].x;
        qs[gr][n].y = __shfl_sync(0xffffffffu, sum[n], 4 * col + 4) * f[gr].y;
      }
      f[gr].x *= 0x1p9f, f[gr].y *= 0x1p9f;  // the codes come times 2^-9
#pragma unroll
      for (int j = 0; j < 2; ++j)
        row_keys(p, a.s, (row0 + kRows * gr + col + j) / p.G, lo[gr][j], hi[gr][j]);
    }
    __syncwarp();
    // keys that every row sees
    int all_lo, all_hi, unused;
    row_keys(p, a.s, p.T - 1, all_lo, unused);
    row_keys(p, a.s, 0, unused, all_hi);

    float acc[RG][MT][4] = {};
    float2 zero_sum[RG][NG] = {}, l[RG] = {}, m[RG], due[RG];
#pragma unroll
    for (int gr = 0; gr < RG; ++gr) {
      m[gr] = make_float2(kLeast, kLeast);
      due[gr] = make_float2(1.f, 1.f);  // what has left acc lies in `state`, to be multiplied by this
    }
    bool kept = false;
    int chain = 0;
    for (int n = 0; n < a.n; ++n) {
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      __syncwarp();
      const uint32_t bad = sh.bad[warp][got];
      const uint32_t base = ring + got * g_::STAGE;
      const int first = (a.s.tile0 + a.i0 + n) * TOK;
#pragma unroll 1
      for (int tok = 0; tok < TOK; tok += 16 * H) {
        const int key0 = first + tok;
        if (key0 >= a.s.hi || key0 + 16 * H <= a.s.lo) continue;
        auto work = [&](auto masked) {
          constexpr bool PART = decltype(masked)::value;
          const uint32_t at = base + tok * RB;  // the first of the keys
          const uint32_t par = base + 2 * g_::CODES + tok * 4 * NG;
          uint32_t kw[H][P][2], kp[H][2][NG], vp[H][2][NG];
#pragma unroll
          for (int h = 0; h < H; ++h) {
#pragma unroll
            for (int i2 = 0; i2 < P / 2; ++i2)
              da::ldsm_x4((at + h * 16 * RB + k_lane) ^ (i2 << 5), kw[h][2 * i2][0], kw[h][2 * i2][1],
                          kw[h][2 * i2 + 1][0], kw[h][2 * i2 + 1][1]);
            load_params<NG>(par + (16 * h + key_a) * 4 * NG, kp[h][0]);
            load_params<NG>(par + (16 * h + key_b) * 4 * NG, kp[h][1]);
            load_params<NG>(par + (TOK + 16 * h + key_a) * 4 * NG, vp[h][0]);
            load_params<NG>(par + (TOK + 16 * h + key_b) * 4 * NG, vp[h][1]);
          }
          // -------------------------------------------- scores
          float2 x[RG][H][2];  // of keys a and b; columns 2c, 2c + 1
          {
            float2 u[RG][H][2], z[RG][H][2];
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              float ah[RG][H][4];
              [[maybe_unused]] float al[RG][H][4];
#pragma unroll
              for (int i2 = n * GP; i2 < (n + 1) * GP; ++i2) {
#pragma unroll
                for (int o2 = 0; o2 < 2; ++o2) {
                  uint32_t q[RG][4];
#pragma unroll
                  for (int gr = 0; gr < RG; ++gr) {
                    const int at = gr * P * 2 + 2 * i2 + o2;
                    q[gr][2] = q[gr][3] = 0;
                    if constexpr (g_::QREG) {
                      q[gr][0] = qf[at][0], q[gr][1] = qf[at][1];
                      if constexpr (!PACK) q[gr][2] = qf[at][2], q[gr][3] = qf[at][3];
                    } else if constexpr (PACK) {
                      const uint2 w = reinterpret_cast<const uint2*>(qfrag)[at * 32 + lane];
                      q[gr][0] = w.x, q[gr][1] = w.y;
                    } else {
                      const uint4 w = qfrag[at * 32 + lane];
                      q[gr][0] = w.x, q[gr][1] = w.y, q[gr][2] = w.z, q[gr][3] = w.w;
                    }
                  }
#pragma unroll
                  for (int h = 0; h < H; ++h) {
                    const uint32_t a0 = kw[h][i2][0], a1 = kw[h][i2][1];
                    const uint32_t f0 = codes2(a0, o2), f1 = codes2(a1, o2);
                    const uint32_t f2 = codes2(a0 >> 8, o2), f3 = codes2(a1 >> 8, o2);
#pragma unroll
                    for (int gr = 0; gr < RG; ++gr) {
                      if (i2 == n * GP && o2 == 0) {
                        mma_first(ah[gr][h], f0, f1, f2, f3, q[gr][0], q[gr][1]);
                        if constexpr (!PACK) mma_first(al[gr][h], f0, f1, f2, f3, q[gr][2], q[gr][3]);
                      } else {
                        mma(ah[gr][h], f0, f1, f2, f3, q[gr][0], q[gr][1]);
                        if constexpr (!PACK) mma(al[gr][h], f0, f1, f2, f3, q[gr][2], q[gr][3]);
                      }
                    }
                  }
                }
              }
#pragma unroll
              for (int h = 0; h < H; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float sk = half_lo(kp[h][k][n]);
                  const float zk = fmaf(8.f, sk, half_hi(kp[h][k][n]));
#pragma unroll
                  for (int gr = 0; gr < RG; ++gr) {
                    float2 t = make_float2(ah[gr][h][2 * k], ah[gr][h][2 * k + 1]);
                    if constexpr (PACK)
                      t = da::add2(t, make_float2(__shfl_xor_sync(0xffffffffu, t.x, 2),
                                                  __shfl_xor_sync(0xffffffffu, t.y, 2)));
                    else
                      t = da::add2(t, make_float2(al[gr][h][2 * k], al[gr][h][2 * k + 1]));
                    float2 &uu = u[gr][h][k], &zz = z[gr][h][k];
                    if (n == 0) {
                      uu = make_float2(t.x * sk, t.y * sk);
                      zz = make_float2(zk * qs[gr][n].x, zk * qs[gr][n].y);
                    } else {
                      uu = make_float2(fmaf(t.x, sk, uu.x), fmaf(t.y, sk, uu.y));
                      zz = make_float2(fmaf(zk, qs[gr][n].x, zz.x), fmaf(zk, qs[gr][n].y, zz.y));
                    }
                  }
                }
            }
#pragma unroll
            for (int gr = 0; gr < RG; ++gr)
#pragma unroll
              for (int h = 0; h < H; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) x[gr][h][k] = da::fma2(u[gr][h][k], f[gr], z[gr][h][k]);
          }
          uint32_t vw[H][P][2];
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i2 = 0; i2 < P / 2; ++i2)
              da::ldsm_b8_x2_trans((at + h * 16 * RB + v_lane) ^ (i2 << 5), vw[h][2 * i2][0],
                                   vw[h][2 * i2][1], vw[h][2 * i2 + 1][0], vw[h][2 * i2 + 1][1]);
          if (p.softcap2 > 0.f) {
#pragma unroll
            for (int gr = 0; gr < RG; ++gr)
#pragma unroll
              for (int h = 0; h < H; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float2& y = x[gr][h][k];
                  y.x = soft_cap(y.x * p.softcap_inv, p.softcap2);
                  y.y = soft_cap(y.y * p.softcap_inv, p.softcap2);
                }
          }
          // -------------------------------------------- masks
          uint32_t seen[RG] = {};
          if constexpr (PART) {
#pragma unroll
            for (int gr = 0; gr < RG; ++gr)
#pragma unroll
              for (int j = 0; j < 4 * H; ++j) {
                const int t = 16 * (j / 4) + (j % 4 < 2 ? key_a : key_b), k = key0 + t;
                float2& y = x[gr][j / 4][j % 4 / 2];
                if (k >= lo[gr][j & 1] && k < hi[gr][j & 1] && !(bad >> ((tok + t) >> p.log2_eb) & 1))
                  seen[gr] |= 1u << j;
                else
                  (j & 1 ? y.y : y.x) = -INFINITY;
              }
          }
          // -------------------------------------------- reference
          float2 top[RG];  // a NaN score leaves it alone
#pragma unroll
          for (int gr = 0; gr < RG; ++gr) top[gr] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t most = vp[h][k][0] & 0x7fffu;
#pragma unroll
              for (int n = 1; n < NG; ++n) most = max(most, vp[h][k][n] & 0x7fffu);
              // exponent of the key's largest value scale: the scale is less than 2^e
              const float e = __uint_as_float(most >> 10 | 0x4b000000u) - (8388608.f + 14.f);
#pragma unroll
              for (int gr = 0; gr < RG; ++gr) {
                top[gr].x = fmaxf(top[gr].x, x[gr][h][k].x + e);
                top[gr].y = fmaxf(top[gr].y, x[gr][h][k].y + e);
              }
            }
          bool past = false;
#pragma unroll
          for (int gr = 0; gr < RG; ++gr)
            past |= top[gr].x > m[gr].x + kSlack || top[gr].y > m[gr].y + kSlack;
          if (__any_sync(0xffffffffu, past)) {
#pragma unroll
            for (int gr = 0; gr < RG; ++gr) {
              float2 by, t = top[gr];
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) {
                t.x = fmaxf(t.x, __shfl_xor_sync(0xffffffffu, t.x, off));
                t.y = fmaxf(t.y, __shfl_xor_sync(0xffffffffu, t.y, off));
              }
              t.x = fmaxf(t.x, m[gr].x), t.y = fmaxf(t.y, m[gr].y);
              by.x = t.x == m[gr].x ? 1.f : da::ex2_ftz(m[gr].x - t.x);
              by.y = t.y == m[gr].y ? 1.f : da::ex2_ftz(m[gr].y - t.y);
              m[gr] = t;
              l[gr] = da::mul2(l[gr], by);
              due[gr] = da::mul2(due[gr], by);
#pragma unroll
              for (int n = 0; n < NG; ++n) zero_sum[gr][n] = da::mul2(zero_sum[gr][n], by);
#pragma unroll
              for (int i2 = 0; i2 < MT; ++i2) {
                acc[gr][i2][0] *= by.x, acc[gr][i2][1] *= by.y;
                acc[gr][i2][2] *= by.x, acc[gr][i2][3] *= by.y;
              }
            }
          }
          // -------------------------------------------- weights
#pragma unroll
          for (int gr = 0; gr < RG; ++gr) {
            const float2 up = make_float2(kShift - m[gr].x, kShift - m[gr].y);
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float2 y = da::add2(x[gr][h][k], up);
                y.x = da::ex2_ftz(y.x), y.y = da::ex2_ftz(y.y);
                if constexpr (PART) {
                  if (!(seen[gr] >> (4 * h + 2 * k) & 1)) y.x = 0.f;
                  if (!(seen[gr] >> (4 * h + 2 * k) & 2)) y.y = 0.f;
                }
                x[gr][h][k] = y;
                l[gr] = da::add2(l[gr], y);
              }
          }
          // -------------------------------------------- values
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            uint32_t ph[RG][H][2], pl[RG][H][2];  // P^T: the two terms
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float sv = half_lo(vp[h][k][n]);
                const float zv = fmaf(8.f, sv, half_hi(vp[h][k][n]));
#pragma unroll
                for (int gr = 0; gr < RG; ++gr) {
                  const float2 y = x[gr][h][k];
                  float2 &zs = zero_sum[gr][n], w = make_float2(y.x * sv, y.y * sv);
                  if constexpr (PART) {  // a key that is not seen may have any scale and zero
                    const bool on0 = seen[gr] >> (4 * h + 2 * k) & 1, on1 = seen[gr] >> (4 * h + 2 * k) & 2;
                    w = make_float2(on0 ? w.x : 0.f, on1 ? w.y : 0.f);
                    zs.x += on0 ? y.x * zv : 0.f;
                    zs.y += on1 ? y.y * zv : 0.f;
                  } else {
                    zs.x = fmaf(y.x, zv, zs.x);
                    zs.y = fmaf(y.y, zv, zs.y);
                  }
                  uint32_t &hi_t = ph[gr][h][k], &lo_t = pl[gr][h][k];
                  da::split_half2(w.x, w.y, hi_t, lo_t);
                  if (PACK && c >= 2) hi_t = lo_t;
                  hi_t = da::movmatrix_trans(hi_t);
                  if constexpr (!PACK) lo_t = da::movmatrix_trans(lo_t);
                }
              }
            // two pieces' products of one term, then of the other: each waits for none before it
            constexpr int PP = GP > 1 ? 2 : 1;
#pragma unroll
            for (int i2 = n * GP; i2 < (n + 1) * GP; i2 += PP)
#pragma unroll
              for (int h = 0; h < H; ++h) {
                uint32_t fr[2 * PP][4];
#pragma unroll
                for (int k = 0; k < 2 * PP; ++k) {
                  const uint32_t a0 = vw[h][i2 + k / 2][0], a1 = vw[h][i2 + k / 2][1];
                  fr[k][0] = codes2(a0, k & 1), fr[k][1] = codes2(a1, k & 1);
                  fr[k][2] = codes2(a0 >> 8, k & 1), fr[k][3] = codes2(a1 >> 8, k & 1);
#pragma unroll
                  for (int gr = 0; gr < RG; ++gr)
                    mma(acc[gr][2 * i2 + k], fr[k][0], fr[k][1], fr[k][2], fr[k][3], ph[gr][h][0],
                        ph[gr][h][1]);
                }
                if constexpr (!PACK) {
#pragma unroll
                  for (int k = 0; k < 2 * PP; ++k)
#pragma unroll
                    for (int gr = 0; gr < RG; ++gr)
                      mma(acc[gr][2 * i2 + k], fr[k][0], fr[k][1], fr[k][2], fr[k][3], pl[gr][h][0],
                          pl[gr][h][1]);
                }
              }
          }
        };
        if (key0 < all_lo || key0 + 16 * H > all_hi || bad) work(std::true_type());
        else work(std::false_type());
      }
      __syncwarp();  // the stage is read
      if (++got == STAGES) got = 0;
      copy(a, n + STAGES);
      if (++chain == chain_keys(PACK) / TOK && n + 1 < a.n) {
#pragma unroll
        for (int gr = 0; gr < RG; ++gr) {
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            float (&y)[4] = acc[gr][i];
            float4 v = make_float4(y[0], y[1], y[2], y[3]), *at = state_at(gr * MT + i);
            if (kept) {
              const float4 w = *at;
              const float2 d = due[gr];
              v = make_float4(fmaf(w.x, d.x, v.x), fmaf(w.y, d.y, v.y), fmaf(w.z, d.x, v.z),
                              fmaf(w.w, d.y, v.w));
            }
            *at = v;
            y[0] = y[1] = y[2] = y[3] = 0.f;
          }
          due[gr] = make_float2(1.f, 1.f);
        }
        kept = true;
        chain = 0;
      }
    }
    // ------------------------------------------------ the part's state
#pragma unroll
    for (int gr = 0; gr < RG; ++gr) {
      float2 sum = l[gr], zs[NG];
#pragma unroll
      for (int n = 0; n < NG; ++n) zs[n] = zero_sum[gr][n];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        sum.x += __shfl_xor_sync(0xffffffffu, sum.x, off);
        sum.y += __shfl_xor_sync(0xffffffffu, sum.y, off);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          zs[n].x += __shfl_xor_sync(0xffffffffu, zs[n].x, off);
          zs[n].y += __shfl_xor_sync(0xffffffffu, zs[n].y, off);
        }
      }
      float* to[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // rows of the lane's columns
        const int own = kRows * gr + col + j, r = row0 + own;
        const float mj = j ? m[gr].y : m[gr].x, lj = j ? sum.y : sum.x;
        to[j] = nullptr;
        if (r >= p.R || (PACK && c >= 2)) continue;
        if (a.slot < 0) {
          const int t = r / p.G, h = a.kv * p.G + (r - t * p.G);
          const long long row = ((long long)a.b * p.T + t) * p.Hq + h;
          to[j] = p.out + row * D;
          if (g == 0 && p.lse) p.lse[row] = lj == 0.f ? -INFINITY : (mj - kShift + log2f(lj)) * kLn2;
        } else {
          const long long row = ((long long)share * 2 + a.slot) * p.unit_rows + rg * WROWS + own;
          to[j] = p.part_o + row * D;
          if (g == 0) p.part_ml[row] = make_float2(mj, lj);
        }
      }
      const float2 by = a.slot < 0 ? make_float2(sum.x == 0.f ? 0.f : 1.f / sum.x,
                                                 sum.y == 0.f ? 0.f : 1.f / sum.y)
                                   : make_float2(1.f, 1.f);
      if (kept) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const float4 w = *state_at(gr * MT + i);
          const float2 d = due[gr];
          float (&y)[4] = acc[gr][i];
          y[0] = fmaf(w.x, d.x, y[0]), y[1] = fmaf(w.y, d.y, y[1]);
          y[2] = fmaf(w.z, d.x, y[2]), y[3] = fmaf(w.w, d.y, y[3]);
        }
      }
      if constexpr (PACK) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[gr][i][j] += __shfl_xor_sync(0xffffffffu, acc[gr][i][j], 2);
      }
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 v = make_float2(acc[gr][2 * i][j], acc[gr][2 * i + 1][j]);
          const float k = j & 1 ? by.y : by.x, z = j & 1 ? zs[i / GP].y : zs[i / GP].x;
          v = da::fma2(v, make_float2(0x1p9f, 0x1p9f), make_float2(z, z));
          if (to[j & 1])
            *reinterpret_cast<float2*>(to[j & 1] + 32 * i + 2 * g + (j & 2 ? 16 : 0)) =
                make_float2(v.x * k, v.y * k);
        }
    }
  }
}

// Adds up the states of units that several shares hold, a warp an output row; rows of sequences without a key
// to see are written here too.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) q4_merge_kernel(const __grid_constant__ Q4Params p) {
  constexpr int V = D / 32;  // values of a lane, side by side
  using Vec = typename std::conditional<V == 2, float2, float4>::type;
  constexpr int N = V == 8 ? 2 : 1;  // vectors of a lane, 128 values apart
  da::wait_for_grid_before();
  da::let_next_grid_start();
  const int lane = threadIdx.x % 32;
  const long long row = (long long)blockIdx.x * kMergeWarps + threadIdx.x / 32;
  if (row >= (long long)p.B * p.T * p.Hq) return;
  const int b = (int)(row / (p.T * p.Hq)), th = (int)(row - (long long)b * p.T * p.Hq);
  const int t = th / p.Hq, h = th - t * p.Hq, kv = h / p.G, r = t * p.G + (h - kv * p.G);
  const int pre0 = p.pre[b], nt = p.pre[b + 1] - pre0, all = p.pre[p.B], upb = p.Hkv * p.blocks;
  Vec* out = reinterpret_cast<Vec*>(p.out + row * D) + lane;
  if (nt == 0) {
    for (int i = 0; i < N; ++i) out[32 * i] = Vec{};
    if (lane == 0 && p.lse) p.lse[row] = -INFINITY;
    return;
  }
  const int unit_rows = p.unit_rows, block = r / unit_rows;
  const Shares shares(all * upb, p.shares);
  const int u0 = pre0 * upb + (kv * p.blocks + block) * nt, u1 = u0 + nt;
  const int s0 = shares.of(u0), s1 = shares.of(u1 - 1);
  if (s0 == s1) return;  // whole
  // the first part is its share's first one if the unit starts there, the others are their shares' first
  const int slot0 = shares.start(s0) == u0 ? 0 : 1;
  auto place = [&](int s) {
    return ((long long)s * 2 + (s == s0 ? slot0 : 0)) * unit_rows + (r - block * unit_rows);
  };
  // the first parts' sums are on their way while the weights are worked out (32 chats of 512 to 4096 keys: 32.5 us, else
  // 34.9)
  constexpr int kAhead = 4;
  auto part = [&](int s) {
    return reinterpret_cast<const Vec*>(p.part_o + place(s) * D) + lane;
  };
  Vec ahead[kAhead][N] = {};
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (s0 + k <= s1) ahead[k][i] = part(s0 + k)[32 * i];
  float top = -INFINITY, l = 0.f;
  for (int s = s0 + lane; s <= s1; s += 32) top = fmaxf(top, p.part_ml[place(s)].x);
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float sum[N][V / N] = {};
  for (int base = s0; base <= s1; base += 32) {
    float mine = 0.f;
    if (base + lane <= s1) {
      const float2 x = p.part_ml[place(base + lane)];
      mine = x.x == top ? 1.f : da::ex2_ftz(x.x - top);
      l = fmaf(mine, x.y, l);
    }
    const int n = min(32, s1 - base + 1);
    auto add = [&](float f, const Vec& v, int i) {
      const float* y = reinterpret_cast<const float*>(&v);
#pragma unroll
      for (int j = 0; j < V / N; ++j) sum[i][j] = fmaf(f, y[j], sum[i][j]);
    };
    int k0 = 0;
    if (base == s0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float f = __shfl_sync(0xffffffffu, mine, k);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (k < n) add(f, ahead[k][i], i);
      }
      k0 = kAhead;
    }
#pragma unroll 4
    for (int k = k0; k < n; ++k) {
      const float f = __shfl_sync(0xffffffffu, mine, k);
#pragma unroll
      for (int i = 0; i < N; ++i) add(f, part(base + k)[32 * i], i);
    }
  }
  for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    Vec v;
    float* y = reinterpret_cast<float*>(&v);
#pragma unroll
    for (int j = 0; j < V / N; ++j) y[j] = sum[i][j] * inv;
    out[32 * i] = v;
  }
  if (lane == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (top - kShift + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------ host
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int warps_of(int D, int rows) {
  return D == 256                ? Geo<256, 2, 8>::WARPS
         : D == 128 && rows == 16 ? Geo<128, 1, 16>::WARPS
                                  : Geo<128, 1, 8>::WARPS;
}

struct Shape {
  int rows, warps;    // query rows of a warp, warps of a unit
  int blocks, chunk;  // units of a kv head, sequences of a launch
};

void set_rows(Shape& s, long long rows, int of_warp) {
  const long long n = of_warp < kRows ? kRows : of_warp, warps = (rows + n - 1) / n;
  s.rows = of_warp;
  s.warps = 1;
  while (s.warps < warps && s.warps < kMaxWarps) s.warps *= 2;
  s.blocks = (int)((warps + s.warps - 1) / s.warps);
}

// 16 rows a warp take less work in all, but leave fewer shares with more latency each: they are for many heads
// with room for long sequences.  D = 128, 16 rows, us with 16 and 8: 512 heads of 2048 to 24,000 keys 283 and 326, 160 of
// 8500 98 and 109, 800 of 100 to 600 49 and 46, 48 of 1000 to 9000 48 and 41.  D = 64, groups of 32 and 64 (the first
// spills 144 bytes with 16 rows): 512 heads of 2048 to 24,000 keys 216 and 245, 174 and 207; 192 of 1000 to 9000 53 and
// 51, 45 and 45; 800 of 100 to 600 43 and 37, 37 and 34.  The room stands for the lengths, which the host does not
// know: short sequences in large tables take the longer form.
void choose_rows(const da_params* p, int q_len, int sms, Shape& s) {
  const long long rows = (long long)q_len * p->num_q_heads / p->num_kv_heads;
  if (rows > 8 && p->head_dim <= 128 && (long long)p->batch * p->num_kv_heads >= sms &&
      (long long)p->max_blocks_per_seq * p->block_size >= 1024)
    set_rows(s, rows, 16);
}

int check(const da_params* p, int group, int q_len, Shape& s) {
  int st = da::check_paged(p);
  if (st == DA_OK) st = da::check_q4(p, group);
  if (st != DA_OK) return st;
  if (q_len < 1) return DA_ERR_INVALID;
  const long long cap = (long long)p->max_blocks_per_seq * p->block_size;
  const long long all_rows = (long long)q_len * p->num_q_heads;
  const long long rows = all_rows / p->num_kv_heads;
  if (cap > 0x7fffffffLL - 1024 || all_rows > 0x7fffffffLL - 1024) return DA_ERR_UNSUPPORTED;
  if (da::q4_page_bytes(p->block_size, p->head_dim, group) * p->num_kv_heads > 0xffffffffLL)
    return DA_ERR_UNSUPPORTED;
  set_rows(s, rows, rows <= 4 ? 4 : 8);
  // tiles and rows of a launch count in 31 bits
  const long long tiles = (cap / (4096 / p->head_dim) + 2) * p->num_kv_heads * s.blocks;
  long long most = (0x7fffffffLL - 4096) / tiles;
  if (most > 0x7fffffffLL / all_rows) most = 0x7fffffffLL / all_rows;
  if (most < 1) return DA_ERR_UNSUPPORTED;
  s.chunk = (int)(most < kMaxBatch ? most : kMaxBatch);
  return DA_OK;
}

struct Layout {
  size_t pre, ml, o, total;
};
Layout layout(int sms, int D, int wrows) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Layout w;
  // two states of each warp's rows
  const size_t rows = (size_t)sms * warps_of(D, wrows) * 2 * (wrows < kRows ? kRows : wrows);
  w.pre = 0;
  w.ml = up((kMaxBatch + 1) * sizeof(int));
  w.o = w.ml + up(rows * sizeof(float2));
  w.total = w.o + up(rows * D * sizeof(float));
  return w;
}

template <int D, int NG, int ROWS>
cudaError_t launch_rows(Q4Params& k, int grid, cudaStream_t s) {
  using g_ = Geo<D, NG, ROWS>;
  static_assert(sizeof(Shared<g_::WARPS, g_::STAGES>) <= 2048, "more than a processor's shared memory");
  cudaError_t err = cudaFuncSetAttribute(q4_kernel<D, NG, ROWS>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, g_::kMost);
  if (err != cudaSuccess) return err;
  k.log2_eb = 0;
  while ((2 << k.log2_eb) <= g_::TOK && k.log2_eb < k.log2_bs) ++k.log2_eb;
  k.shares = grid * (g_::WARPS / k.warps);
  err = da::launch_early(q4_kernel<D, NG, ROWS>, grid, g_::THREADS, g_::SMEM + (k.B + 1) * 4, s, k);
  if (err != cudaSuccess) return err;
  const long long rows = (long long)k.B * k.T * k.Hq;
  return da::launch_early(q4_merge_kernel<D>, (unsigned)((rows + kMergeWarps - 1) / kMergeWarps),
                          32 * kMergeWarps, 0, s, k);
}

template <int D, int NG>
cudaError_t launch(Q4Params& k, int rows, int grid, cudaStream_t s) {
  if constexpr (D <= 128)
    if (rows == 16) return launch_rows<D, NG, 16>(k, grid, s);
  return rows == 4 ? launch_rows<D, NG, 4>(k, grid, s) : launch_rows<D, NG, 8>(k, grid, s);
}

cudaError_t launch(Q4Params& k, int D, int group, int rows, int grid, cudaStream_t s) {
  switch (D * 1000 + group) {
    case 64032: return launch<64, 2>(k, rows, grid, s);
    case 64064: return launch<64, 1>(k, rows, grid, s);
    case 128032: return launch<128, 4>(k, rows, grid, s);
    case 128064: return launch<128, 2>(k, rows, grid, s);
    case 128128: return launch<128, 1>(k, rows, grid, s);
    case 256032: return launch<256, 8>(k, rows, grid, s);
    case 256064: return launch<256, 4>(k, rows, grid, s);
    default: return launch<256, 2>(k, rows, grid, s);
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
  choose_rows(p, q_len, sms, s);
  return layout(sms, p->head_dim, s.rows).total;
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
  choose_rows(p, q_len, sms, shape);
  const Layout w = layout(sms, p->head_dim, shape.rows);
  if (!workspace || workspace_bytes < w.total) return DA_ERR_WORKSPACE;
  Q4Params k = {};
  k.pool = pool;
  k.dev_status = dev_status;
  k.T = q_len;
  k.G = p->num_q_heads / p->num_kv_heads;
  k.R = k.T * k.G;
  k.Hq = p->num_q_heads;
  k.Hkv = p->num_kv_heads;
  while ((1 << k.log2_bs) < p->block_size) ++k.log2_bs;
  k.max_blocks = p->max_blocks_per_seq;
  k.num_blocks = p->num_blocks;
  k.window = p->sliding_window;
  k.causal = p->causal;
  k.warps = shape.warps;
  k.blocks = shape.blocks;
  k.unit_rows = shape.warps * (shape.rows < kRows ? kRows : shape.rows);
  k.qscale = da::base2_scale(p);
  // cap and reciprocal are finite for the largest and the least caps too: a score of 0 stays 0
  constexpr float kMostF32 = 3.402823466e38f;
  k.softcap2 = fminf(p->softcap * 1.4426950408889634f, kMostF32);
  k.softcap_inv = k.softcap2 > 0.f ? (float)fmin(1.0 / (double)k.softcap2, kMostF32) : 0.f;
  k.page_bytes = da::q4_page_bytes(p->block_size, p->head_dim, group);
  k.stride = (uint32_t)(k.page_bytes * p->num_kv_heads);
  char* ws = static_cast<char*>(workspace);
  k.pre = reinterpret_cast<int*>(ws + w.pre);
  k.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  k.part_o = reinterpret_cast<float*>(ws + w.o);
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
    if (launch(k, p->head_dim, group, shape.rows, sms, static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return DA_ERR_CUDA;
  }
  return DA_OK;
}

}  // extern "C"
