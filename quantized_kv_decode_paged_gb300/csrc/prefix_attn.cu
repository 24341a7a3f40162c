// prefix_attn.cu — decode attention of a batch that shares the pages of a
// long prefix.
//
// Row (b, t, h) attends to the keys [lo, hi) its masks leave: softmax over
// s_j = scale <q, k_j> (softcap on top), out = sum p_j v_j / sum p_j and
// lse = m + ln sum e^(s_j - m), kept as the running state (m, l, o) of one
// pass over the keys in base-2 units.
//
// Work.  The rows of one kv head (sequences x query tokens x its query
// heads) that share keys are cut into tiles of 128 rows, the keys into tiles
// of 128 (64 for D = 256).  A prefix unit is a (kv head, tile of the batch's
// rows) over the prefix, an own unit a (sequence, kv head, tile of its rows)
// over its own keys.  All units' key tiles form one list; every CTA takes an
// equal run of it (tiles cost the same: the MMA's M is 128 whether a tile has
// 4 rows or 128).  A unit that lies in one CTA leaves its state in
// the row's place; the parts of a unit that CTA boundaries cut go to the
// CTAs' slots.  prefix_merge_kernel joins a row's states:
// M = max m_s, w_s = 2^(m_s - M), out = sum w_s o_s / sum w_s l_s.
//
// A tile.  S = Q K^T and O_tile = P V run on the tensor cores (tcgen05), f16
// operands and f32 accumulators in tensor memory.  Q (f32) is held as
// two f16 terms of q / 2^e, e the row's exponent, P as two f16 terms: 22 bits
// each, so out keeps f32's accuracy (one term would leave 2^-12).  That doubles
// the products: 8 * 128 * D flops a key; a 128-key tile of D = 128 is 2048
// cycles of the tensor pipe for 64 KB of K and V, about the rate at which
// HBM delivers them.  The tensor cores' f32 sums truncate: a long chain of
// them drifts (2^-24 of the sum a step on average; 3.6e-5 of the result after 145 tiles
// in one accumulator).  So every tile starts a new accumulator, the low terms go first
// (their steps truncate at their own size), and the sums over tiles are ordinary f32 adds in
// registers.
//
// Warps.  0: TMA of K and V pages into a ring of tiles.  1: one thread issues
// the products, QK(x + 2) behind PV(x), so that the tensor pipe works on later
// tiles' scores while the softmax of one runs (S and P share three buffers).  2, 3: the next
// unit's Q, when its rows are few.  4-7, softmax: one thread a row, scores to weights, running
// maximum and sum.  8-11 (and 12-15 for D = 256, 128 columns each), sums:
// one thread a row, acc = acc * 2^(m_old - m_new) + O_tile, and the state's store.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/decode_attn.h"
#include "launch.h"
#include "ptx.cuh"
#include "tc5.cuh"

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

// ------------------------------------------------------------------ what a row sees
// Length of sequence b (clamped to its table; 0 when its query position is
// negative: it sees nothing) and position of its first query token.
// Returns device-status bits.
__device__ __forceinline__ int seq_info(const PrefixParams& p, int b, int& len, int& qp) {
  int flags = 0;
  const int cap = p.max_blocks * p.bs;
  len = p.seq_lens[b];
  if (len < 0 || len > cap) {
    flags |= DEV_BAD_SEQ_LEN;
    len = len < 0 ? 0 : cap;
  }
  qp = len - p.T;
  if (p.q_pos) {
    qp = p.q_pos[b];
    if (qp < 0) {
      flags |= DEV_BAD_QPOS;
      len = 0;
    }
  }
  return flags;
}

// Keys [lo, hi) that the query tokens t0 .. t1 see between them: token t0's
// lower bound, token t1's upper bound.
__device__ __forceinline__ void key_range(const PrefixParams& p, int len, int qp, int t0, int t1,
                                          int& lo, int& hi) {
  const long long a = (long long)qp + t0, z = (long long)qp + t1 + 1;
  const long long l = (p.window > 0 && a >= p.window) ? a - p.window + 1 : 0;
  const long long h = p.causal && z < len ? z : len;
  lo = hi = 0;
  if (h > l) {
    lo = (int)l;
    hi = (int)h;
  }
}

// Page of key k of sequence b (not checked against num_blocks).
__device__ __forceinline__ int page_of(const PrefixParams& p, int b, int k) {
  const int c = k >> p.log2_bs;
  return c < p.prefix_pages ? p.prefix_table[c]
                            : p.block_table[(long long)b * p.max_blocks + c];
}

// One warp's state of a row over keys [k0, k1), key by key: lane i holds the
// values [i * D/32, (i + 1) * D/32) of q and o.  Pages outside the pool are masked.
template <int D>
__device__ void attend_row(const PrefixParams& p, int b, int kv, const float (&q)[D / 32], int k0,
                           int k1, float& m, float& l, float (&o)[D / 32]) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  m = -kInf;
  l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int k = k0; k < k1; ++k) {
    const int blk = page_of(p, b, k);
    if (blk < 0 || blk >= p.num_blocks) continue;
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
}

// ------------------------------------------------------------------ geometry
template <int D>
struct PGeo {
  static constexpr int KT = prefix_tile_keys(D);
  static constexpr int SL = D / 64;               // 128-byte slices of a row
  static constexpr int TILE = KT * D * 2;         // bytes of a K or V tile
  static constexpr int QTERM = kPrefixRows * D * 2;  // bytes of one term of Q
  static constexpr int RING = D == 64 ? 8 : D == 128 ? 4 : 3;  // K and V tiles in flight
  static constexpr int NS = 3;                    // S / P buffers
  static constexpr int S0 = D;                    // tensor-memory columns: O, then S / P
  static constexpr int F0 = S0 + NS * KT;         // then, if any are left, the factors
  static constexpr bool FAC_TMEM = F0 + NS <= 512;
  static constexpr int AC = D < 128 ? D : 128;    // columns a sum thread holds
  static constexpr int SUMG = D / AC;             // sum warpgroups
  static constexpr int THREADS = 256 + 128 * SUMG;
  // Registers a thread: at launch, then by role (setmaxnreg); the roles'
  // sum over the warpgroups stays within the launch's.
  static constexpr int REG_LAUNCH = SUMG == 1 ? 168 : 128;
  static constexpr int REG_LOAD = SUMG == 1 ? 72 : 64;
  static constexpr int REG_SOFT = SUMG == 1 ? 232 : 128;
  static constexpr int REG_SUM = SUMG == 1 ? 200 : 160;
  static_assert(F0 <= 512, "tensor memory");
  static_assert(REG_LOAD + REG_SOFT + SUMG * REG_SUM <= (2 + SUMG) * REG_LAUNCH, "registers");
  static_assert(THREADS * REG_LAUNCH <= 65536, "registers");
};

constexpr int kSmallRows = 64;  // parts of at most this many rows share the Q buffer in halves
// Weights are kept times 2^10: those down to 2^-24 of a row's largest stay normal f16
// numbers, and the largest is far from f16's limit.
constexpr float kShift = 10.f;

template <int D>
struct PrefixSmem {
  using G = PGeo<D>;
  static constexpr int MAXB = prefix_max_batch(D);
  uint8_t q[2 * G::QTERM];
  uint8_t ring[G::RING * G::TILE];
  uint64_t full[G::RING], empty[G::RING];
  uint64_t s_full[G::NS], p_full[G::NS], pv_done[G::NS];
  uint64_t o_free, q_full[2], q_free[2], drain;
  float row_scale[kPrefixRows];                          // qscale * 2^e, by row of the Q buffer
  float fac[G::FAC_TMEM ? 1 : G::NS * kPrefixRows];      // 2^(m_old - m_new) of a tile's rows
  int cum[MAXB + 1];                                     // own-key tiles before sequence b
  int len[MAXB], qp[MAXB];                               // seq_info
  int bad[8];                                            // per tile (mod 8): masked boxes of keys
  int warp_sum[16];
  int lo, hi;                                            // prefix keys some row sees
  int abort;
  uint32_t tmem;
};
static_assert(sizeof(PrefixSmem<64>) <= kSmemLimit && sizeof(PrefixSmem<128>) <= kSmemLimit &&
                  sizeof(PrefixSmem<256>) <= kSmemLimit,
              "shared memory");

__device__ __forceinline__ long long part_start(int c, long long total, int ctas) {
  return (long long)c * total / ctas;
}
// The CTA whose run holds tile g.
__device__ __forceinline__ int part_cta(long long g, long long total, int ctas) {
  return (int)(((g + 1) * ctas - 1) / total);
}

// The parts of units that a CTA's run [g0, g1) of the tile list is made of,
// one after the other.  Part: rows [r0, r0 + nr) of kv head h (r0 counts the
// batch's rows in the prefix, the sequence's in its own keys), key tiles
// [i0, i0 + n), tile i's keys starting at base + i * KT.
template <int D>
struct Cursor {
  static constexpr int KT = PGeo<D>::KT;
  const PrefixParams& p;
  const PrefixSmem<D>& s;
  long long left;        // tiles of the run from this part on
  int P, pn;             // prefix keys; tiles of a prefix unit
  int k = 0;             // parts so far
  int h, b, rt;          // b < 0: prefix; rt: tile of rows
  int r0, nr;
  int base, klo, khi;    // keys [klo, khi) may be seen
  int unit_n, i0, n;

  __device__ __forceinline__ Cursor(const PrefixParams& p_, const PrefixSmem<D>& s_, long long tp,
                                    long long g0, long long g1)
      : p(p_), s(s_), left(g1 - g0), P(p_.prefix_pages << p_.log2_bs) {
    const int pt0 = s.lo / KT;
    pn = s.hi > s.lo ? (s.hi + KT - 1) / KT - pt0 : 0;
    h = b = rt = r0 = nr = base = klo = khi = unit_n = i0 = n = 0;
    if (left <= 0) return;
    if (g0 < tp) {
      const int u = (int)(g0 / pn);
      i0 = (int)(g0 - (long long)u * pn);
      h = u / p.row_tiles;
      rt = u - h * p.row_tiles;
      b = -1;
    } else {
      const int units1 = p.Hkv * p.own_tiles;
      const long long x = (g0 - tp) / units1;  // sequence b holds it: cum[b] <= x < cum[b + 1]
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.cum[mid] <= x)
          lo = mid;
        else
          hi = mid;
      }
      b = lo;
      const long long in = g0 - tp - (long long)s.cum[lo] * units1;
      const int each = s.cum[lo + 1] - s.cum[lo];
      const int u = (int)(in / each);
      i0 = (int)(in - (long long)u * each);
      h = u / p.own_tiles;
      rt = u - h * p.own_tiles;
    }
    enter();
  }
  __device__ __forceinline__ bool done() const { return left <= 0; }
  __device__ __forceinline__ bool whole() const { return n == unit_n; }
  // Geometry of the part at (b, h, rt), its first tile i0.
  __device__ __forceinline__ void enter() {
    r0 = rt * kPrefixRows;
    if (b < 0) {
      nr = min(kPrefixRows, p.B * p.R1 - r0);
      klo = s.lo;
      khi = s.hi;
      base = klo / KT * KT;
      unit_n = pn;
    } else {
      nr = min(kPrefixRows, p.R1 - r0);
      key_range(p, s.len[b], s.qp[b], 0, p.T - 1, klo, khi);
      klo = max(klo, P);
      base = P + (klo - P) / KT * KT;
      unit_n = s.cum[b + 1] - s.cum[b];
    }
    n = (int)min((long long)(unit_n - i0), left);
  }
  __device__ __forceinline__ void next() {
    left -= n;
    ++k;
    i0 = 0;
    if (left <= 0) return;
    if (++rt == (b < 0 ? p.row_tiles : p.own_tiles)) {
      rt = 0;
      if (++h == p.Hkv) {
        h = 0;
        b = max(b, -1) + 1;
        while (s.cum[b + 1] == s.cum[b]) ++b;
      }
    }
    enter();
  }
  __device__ __forceinline__ bool small() const { return nr <= kSmallRows; }
  // First row of the Q buffer that the part's rows take.
  __device__ __forceinline__ int q_row() const { return small() ? (k & 1) * kSmallRows : 0; }
  // Sequence, query token and place in [B, T, Hq] of the part's row i.
  __device__ __forceinline__ int out_row(int i, int& seq, int& tok) const {
    int r = r0 + i;
    seq = b;
    if (b < 0) {
      seq = r / p.R1;
      r -= seq * p.R1;
    }
    tok = r / p.G;
    return (seq * p.T + tok) * p.Hq + h * p.G + (r - tok * p.G);
  }
};

// Lengths and positions into shared memory, the tiles of every sequence's own
// keys (running sums) and the prefix keys that some row sees.  All threads
// call it; one thread a sequence.
template <int D>
__device__ int make_plan(const PrefixParams& p, PrefixSmem<D>& s) {
  constexpr int KT = PGeo<D>::KT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = p.prefix_pages << p.log2_bs;
  int n = 0, flags = 0;
  if (tid < p.B) {
    int len, qp, lo, hi;
    flags = seq_info(p, tid, len, qp);
    s.len[tid] = len;
    s.qp[tid] = qp;
    key_range(p, len, qp, 0, p.T - 1, lo, hi);
    if (hi > lo && lo < P) {
      atomicMin(&s.lo, lo);
      atomicMax(&s.hi, min(hi, P));
    }
    const int l = max(lo, P);
    if (hi > l) n = (hi - P + KT - 1) / KT - (l - P) / KT;
  }
  int sum = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += x;
  }
  if (lane == 31) s.warp_sum[warp] = sum;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
  if (tid < p.B) s.cum[tid + 1] = before + sum;
  if (tid == 0) s.cum[0] = 0;
  __syncthreads();
  return flags;
}

// A wait that gives up sets the abort flag; every role then leaves its loop.
template <int D>
__device__ __forceinline__ bool wait_or_abort(const PrefixParams& p, PrefixSmem<D>& s,
                                              uint64_t* bar, uint32_t parity) {
  if (mbar_wait(bar, parity, &s.abort, p.wait_ns)) return true;
  *(volatile int*)&s.abort = 1;
  if (p.dev_status) atomicOr(p.dev_status, DEV_TIMEOUT);
  return false;
}
// The same for all lanes of a warp, which go on or leave together.
template <int D>
__device__ __forceinline__ bool warp_wait(const PrefixParams& p, PrefixSmem<D>& s, uint64_t* bar,
                                          uint32_t parity) {
  return __all_sync(0xffffffffu, wait_or_abort<D>(p, s, bar, parity));
}

// ------------------------------------------------------------------ TMA warp
// K and V tiles into the ring in the order the products take them:
// K(0) K(1) V(0) K(2) V(1) ...  Each lane copies one box.  Boxes without a
// visible key and pages outside the pool are filled with zeros by a copy that
// starts past the pool's last row.
template <int D>
struct Loader {
  using G = PGeo<D>;
  const PrefixParams& p;
  PrefixSmem<D>& s;
  int nsl, sub, slice, boxes;
  int r = 0;  // ring tiles issued
  int flags = 0;

  __device__ __forceinline__ Loader(const PrefixParams& p_, PrefixSmem<D>& s_) : p(p_), s(s_) {
    const int lane = threadIdx.x & 31;
    nsl = G::SL / p.box_slices;
    boxes = G::KT / p.box_rows * nsl;
    sub = lane / nsl;
    slice = lane - sub * nsl;
    if (lane >= boxes) sub = -1;
  }
  // Block id of this lane's box in tile j of the cursor's part (the load may
  // run ahead of its use); num_blocks: no key of it is seen.
  __device__ __forceinline__ int block(const Cursor<D>& c, int j) const {
    const int k0 = c.base + (c.i0 + j) * G::KT + sub * p.box_rows;
    if (sub < 0 || k0 >= c.khi || k0 + p.box_rows <= c.klo) return p.num_blocks;
    const int col = k0 >> p.log2_bs;
    const int blk = c.b < 0 ? p.prefix_table[col]
                            : p.block_table[(long long)c.b * p.max_blocks + col];
    return blk == p.num_blocks ? -1 : blk;
  }
  // x: the tile's number in the CTA's run.
  __device__ __forceinline__ bool issue(const Cursor<D>& c, int j, int x, int blk, bool is_v) {
    const int lane = threadIdx.x & 31, slot = r % G::RING;
    if (r >= G::RING && !warp_wait<D>(p, s, &s.empty[slot], (r / G::RING - 1) & 1)) return false;
    const int k0 = c.base + (c.i0 + j) * G::KT + sub * p.box_rows;
    int row = p.num_blocks << p.log2_bs;
    const bool bad = blk < 0 || blk > p.num_blocks;
    if (!bad && blk < p.num_blocks) row = (blk << p.log2_bs) + (k0 & (p.bs - 1));
    if (!is_v) {
      const int mask = __reduce_or_sync(0xffffffffu, bad ? 1 << sub : 0);
      if (lane == 0) s.bad[x & 7] = mask;
      if (bad) flags |= DEV_BAD_BLOCK;
    }
    // test hook: the first tile of CTA 0 never arrives and its consumer's wait runs out
    const bool skip = p.test_skip_arm && blockIdx.x == 0 && r == 0;
    if (lane == 0 && !skip) mbar_arrive_expect_tx(&s.full[slot], G::TILE);
    __syncwarp();
    if (sub >= 0 && !skip)
      tma_load_4d(s.ring + slot * G::TILE + slice * (G::KT * 128) + sub * p.box_rows * 128,
                  is_v ? &p.tm_v : &p.tm_k, &s.full[slot], 0, row, slice, c.h);
    ++r;
    return true;
  }
  __device__ __forceinline__ void run(long long tp, long long g0, long long g1) {
    Cursor<D> ck(p, s, tp, g0, g1), cv = ck;
    const int tiles = (int)(g1 - g0);
    int jk = 0, jv = 0, blk = ck.done() ? 0 : block(ck, 0);
    auto next_k = [&](int x) {  // K of tile x; its block id was fetched a step ago
      if (x >= tiles) return true;
      const int now = blk;
      const Cursor<D> c = ck;
      const int j = jk;
      if (++jk == ck.n) {
        jk = 0;
        ck.next();
      }
      if (!ck.done()) blk = block(ck, jk);
      return issue(c, j, x, now, false);
    };
    if (!next_k(0) || !next_k(1)) return;
    for (int x = 0; x < tiles; ++x) {
      if (!issue(cv, jv, x, block(cv, jv), true)) return;
      if (++jv == cv.n) {
        jv = 0;
        cv.next();
      }
      if (!next_k(x + 2)) return;
    }
  }
};

// ------------------------------------------------------------------ Q
// Rows [first, last) of a part's Q into shared memory by one warp: the power
// of two that brings a row's largest value to [2^9, 2^10), then two f16 terms.
template <int D>
__device__ void load_q_rows(const PrefixParams& p, PrefixSmem<D>& s, const Cursor<D>& c, int first,
                            int last) {
  constexpr int V = D / 32;  // values of a lane
  constexpr int BATCH = D >= 256 ? 4 : 8;
  const int lane = threadIdx.x & 31;
  for (int i0 = first; i0 < last; i0 += 32) {
    int seq, tok;
    const int mine = i0 + lane < last ? c.out_row(i0 + lane, seq, tok) : 0;
    for (int u0 = 0; u0 < min(32, last - i0); u0 += BATCH) {
      float x[BATCH][V];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        // rows past the last one repeat it
        const int at = __shfl_sync(0xffffffffu, mine, min(u0 + u, last - i0 - 1));
        const float* src = p.q + (long long)at * D + lane * V;
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 f = *reinterpret_cast<const float2*>(src + i);
          x[u][i] = f.x;
          x[u][i + 1] = f.y;
        }
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const int row = c.q_row() + min(i0 + u0 + u, last - 1);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(x[u][i]));
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        // exponent of the largest value, clamped so that both powers are normal
        int e = (int)(__float_as_uint(m) >> 23) - 127;
        e = min(max(e, -100), 120);
        const float f = __uint_as_float((uint32_t)(9 - e + 127) << 23);
        if (lane == 0) s.row_scale[row] = p.qscale * __uint_as_float((uint32_t)(e - 9 + 127) << 23);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          uint32_t hi, lo;
          split_half2(x[u][i] * f, x[u][i + 1] * f, hi, lo);
          const int d = lane * V + i;
          const int at = (d >> 6) * (kPrefixRows * 128) + row * 128 +
                         ((((d & 63) >> 3) ^ (row & 7)) << 4) + (d & 7) * 2;
          *reinterpret_cast<uint32_t*>(s.q + at) = hi;
          *reinterpret_cast<uint32_t*>(s.q + PGeo<D>::QTERM + at) = lo;
        }
      }
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Warps 2 and 3: Q of the parts with few rows, one part ahead of the products.
template <int D>
__device__ void q_loop(const PrefixParams& p, PrefixSmem<D>& s, long long tp, long long g0,
                       long long g1) {
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 2;
  bool prev_small = true;
  for (Cursor<D> c(p, s, tp, g0, g1); !c.done(); c.next()) {
    const int k = c.k;
    if (c.small()) {
      // the half's last user, and a part of many rows just before
      if (k >= 2 && !warp_wait<D>(p, s, &s.q_free[k & 1], ((k - 2) >> 1) & 1)) return;
      if (!prev_small && !warp_wait<D>(p, s, &s.q_free[(k - 1) & 1], ((k - 1) >> 1) & 1)) return;
      const int half = (c.nr + 1) / 2;
      load_q_rows<D>(p, s, c, w * half, min(c.nr, (w + 1) * half));
      if (lane < 2) mbar_arrive(&s.q_full[k & 1]);  // two of the barrier's four
    }
    prev_small = c.small();
  }
}

// ------------------------------------------------------------------ softmax warps
template <int D, bool CAP>
__device__ void softmax_loop(const PrefixParams& p, PrefixSmem<D>& s, long long tp, long long g0,
                             long long g1) {
  using G = PGeo<D>;
  constexpr int KT = G::KT;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const int row = w * 32 + lane;
  const uint32_t lanes = s.tmem + ((uint32_t)(w * 32) << 16);
  const int box_shift = __ffs(p.box_rows) - 1;
  int x = 0;  // tiles so far
  for (Cursor<D> c(p, s, tp, g0, g1); !c.done(); c.next()) {
    const int k = c.k;
    if (!c.small()) {
      // many rows: they take the whole buffer
      if (k >= 1 && !warp_wait<D>(p, s, &s.q_free[(k - 1) & 1], ((k - 1) >> 1) & 1)) return;
      load_q_rows<D>(p, s, c, min(c.nr, w * 32), min(c.nr, w * 32 + 32));
      if (lane == 0) mbar_arrive(&s.q_full[k & 1]);
    }
    const bool any = w * 32 < c.nr;  // rows of this warp
    const bool on = row < c.nr;
    int lo = 0, hi = 0, orow = 0;
    if (on) {
      int b, tok;
      orow = c.out_row(row, b, tok);
      key_range(p, s.len[b], s.qp[b], tok, tok, lo, hi);
      if (c.b < 0)
        hi = min(hi, c.P);
      else
        lo = max(lo, c.P);
    }
    float scale = 0.f, m = -kInf, l = 0.f;
    bool partial = false;
    for (int j = 0; j < c.n; ++j, ++x) {
      const int buf = x % G::NS;
      if (!warp_wait<D>(p, s, &s.s_full[buf], (x / G::NS) & 1)) return;
      if (j == 0) {
        if (on) scale = s.row_scale[c.q_row() + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.q_free[k & 1]);
      }
      if (any) {
        tc5_fence_after();
        const uint32_t sa = lanes + G::S0 + buf * KT;
        const int k0 = c.base + (c.i0 + j) * KT;
        const int bad = s.bad[x & 7];
        const bool masked =
            !__all_sync(0xffffffffu, (!on || (lo <= k0 && hi >= k0 + KT)) && bad == 0);
        partial |= masked;
        // Two passes over the scores, 32 columns at a time: a loop that stays in the
        // instruction cache and needs few registers.
        float top = m;
#pragma unroll 1
        for (int i0 = 0; i0 < KT; i0 += 32) {
          float v[32];
          tmem_ld32(sa + i0, v);
          tmem_wait_ld();
          tmem_loaded32(v);
          if (CAP || masked) {
            if (CAP) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = capped(v[i] * scale, p.softcap2, p.softcap_inv);
            }
            if (masked) {
              const int a = lo - k0 - i0, z = hi - k0 - i0;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < a || i >= z || ((bad >> ((i0 + i) >> box_shift)) & 1)) v[i] = -kInf;
            }
            tmem_st32(sa + i0, v);
          }
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = v[i];
#pragma unroll
          for (int i = 4; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], v[i]);
          top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (CAP ? 1.f : scale));
        }
        if (CAP || masked) tmem_wait_st();
        // no key so far: any finite reference does
        const float ref = top == -kInf ? 0.f : top;
        const float f = ex2_ftz(m - ref);
        m = top;
        if constexpr (G::FAC_TMEM)
          tmem_st1(lanes + G::F0 + buf, f);
        else
          s.fac[buf * kPrefixRows + row] = f;
        const float cc = CAP ? 1.f : scale, base = ref - kShift;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int i0 = 0; i0 < KT; i0 += 32) {
          float v[32];
          uint32_t ph[16], pl[16];
          tmem_ld32(sa + i0, v);
          tmem_wait_ld();
          tmem_loaded32(v);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float p0 = ex2_ftz(fmaf(v[i], cc, -base));
            const float p1 = ex2_ftz(fmaf(v[i + 1], cc, -base));
            sum[i & 2] += p0;
            sum[(i & 2) + 1] += p1;
            split_half2(p0, p1, ph[i / 2], pl[i / 2]);
          }
          // the weights of 32 keys take the columns of their scores: 16 of high terms, 16 of low
          tmem_st16(sa + i0, ph);
          tmem_st16(sa + i0 + 16, pl);
        }
        l = fmaf(l, f, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        tmem_wait_st();
        tc5_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.p_full[buf]);
    }
    if (on) {
      float2* dst;
      if (!c.whole())
        dst = p.ws_cut_ml + (blockIdx.x * 2 + (k == 0 ? 0 : 1)) * kPrefixRows + row;
      else if (c.b < 0)
        dst = p.ws_pre_ml + orow;
      else
        dst = p.ws_own_ml + orow;
      *dst = make_float2(m - kShift, partial ? -l : l);
    }
  }
}

// ------------------------------------------------------------------ sum warps
template <int D>
__device__ void sum_loop(const PrefixParams& p, PrefixSmem<D>& s, long long tp, long long g0,
                         long long g1) {
  using G = PGeo<D>;
  constexpr int C = G::AC;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const int row = w * 32 + lane, col = ((int)(threadIdx.x >> 7) - 2) * C;
  const uint32_t lanes = s.tmem + ((uint32_t)(w * 32) << 16);
  int x = 0;
  for (Cursor<D> c(p, s, tp, g0, g1); !c.done(); c.next()) {
    const bool any = w * 32 < c.nr, on = row < c.nr;
    float acc[C];
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = 0.f;
    for (int j = 0; j < c.n; ++j, ++x) {
      const int buf = x % G::NS;
      const uint32_t parity = (x / G::NS) & 1;
      if (!warp_wait<D>(p, s, &s.p_full[buf], parity)) return;
      float f = 0.f;
      if (any) {
        if constexpr (G::FAC_TMEM) {
          tc5_fence_after();
          f = tmem_ld1(lanes + G::F0 + buf);
        } else {
          f = s.fac[buf * kPrefixRows + row];
        }
      }
      if (!warp_wait<D>(p, s, &s.pv_done[buf], parity)) return;
      if (any) {
        tc5_fence_after();
        if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
          for (int i = 0; i < C; ++i) acc[i] *= f;
        }
#pragma unroll
        for (int i = 0; i < C; i += 16) {
          float o[16];
          tmem_load16(lanes + col + i, o);
#pragma unroll
          for (int u = 0; u < 16; ++u) acc[i + u] += o[u];
        }
        tc5_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_free);
    }
    if (on) {
      float* dst;
      if (!c.whole()) {
        dst = p.ws_cut_o + ((long long)(blockIdx.x * 2 + (c.k == 0 ? 0 : 1)) * kPrefixRows + row) * D;
      } else {
        int b, tok;
        dst = (c.b < 0 ? p.ws_pre_o : p.out) + (long long)c.out_row(row, b, tok) * D;
      }
#pragma unroll
      for (int i = 0; i < C; i += 4)
        *reinterpret_cast<float4*>(dst + col + i) =
            make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    }
  }
}

// ------------------------------------------------------------------ MMA thread
template <int D>
__device__ void mma_loop(const PrefixParams& p, PrefixSmem<D>& s, long long tp, long long g0,
                         long long g1) {
  using G = PGeo<D>;
  constexpr int KT = G::KT;
  constexpr uint32_t id_qk = f16_idesc(KT, false), id_pv = f16_idesc(D, true);
  const uint32_t tm = s.tmem, q0 = smem_u32(s.q), ring = smem_u32(s.ring);
  Cursor<D> c(p, s, tp, g0, g1);  // of the scores
  const int tiles = (int)(g1 - g0);
  int r = 0;  // ring tiles taken
  int jq = 0;
  auto qk = [&](int y) {  // scores of tile y; the low term first: its steps truncate at its size
    if (y >= tiles) return true;
    const int slot = r % G::RING, buf = y % G::NS;
    if (jq == 0 && !wait_or_abort<D>(p, s, &s.q_full[c.k & 1], (c.k >> 1) & 1)) return false;
    if (y >= G::NS && !wait_or_abort<D>(p, s, &s.pv_done[buf], (y / G::NS - 1) & 1)) return false;
    if (!wait_or_abort<D>(p, s, &s.full[slot], (r / G::RING) & 1)) return false;
    tc5_fence_after();
    const uint32_t k = ring + slot * G::TILE, q = q0 + c.q_row() * 128;
#pragma unroll
    for (int term = 1; term >= 0; --term)
#pragma unroll
      for (int d = 0; d < D; d += 16)
        mma_ss(tm + G::S0 + buf * KT,
               smem_desc(q + term * G::QTERM + (d >> 6) * (kPrefixRows * 128) + (d & 63) * 2, 16,
                         1024),
               smem_desc(k + (d >> 6) * (KT * 128) + (d & 63) * 2, 16, 1024), id_qk,
               term == 0 || d > 0);
    mma_commit(&s.empty[slot]);
    mma_commit(&s.s_full[buf]);
    ++r;
    if (++jq == c.n) {
      jq = 0;
      mma_commit(&s.q_free[c.k & 1]);
      c.next();
    }
    return true;
  };
  if (!qk(0) || !qk(1)) return;
  for (int x = 0; x < tiles; ++x) {
    const int buf = x % G::NS, slot = r % G::RING;
    if (!wait_or_abort<D>(p, s, &s.full[slot], (r / G::RING) & 1)) return;
    if (!wait_or_abort<D>(p, s, &s.p_full[buf], (x / G::NS) & 1)) return;
    if (x > 0 && !wait_or_abort<D>(p, s, &s.o_free, (x - 1) & 1)) return;
    tc5_fence_after();
    const uint32_t v = ring + slot * G::TILE;
#pragma unroll
    for (int term = 1; term >= 0; --term)
#pragma unroll
      for (int k = 0; k < KT; k += 16)
        mma_ts(tm, tm + G::S0 + buf * KT + k / 32 * 32 + term * 16 + k % 32 / 2,
               smem_desc(v + k * 128, KT * 128, 1024), id_pv, term == 0 || k > 0);
    mma_commit(&s.empty[slot]);
    mma_commit(&s.pv_done[buf]);
    ++r;
    if (!qk(x + 2)) return;
  }
}

template <int D, bool CAP>
__global__ void __launch_bounds__(PGeo<D>::THREADS, 1)
    prefix_attn_kernel(const __grid_constant__ PrefixParams p) {
  using G = PGeo<D>;
  extern __shared__ __align__(1024) uint8_t dyn[];
  PrefixSmem<D>& s = *reinterpret_cast<PrefixSmem<D>*>(dyn);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < G::RING; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < G::NS; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 4);
      mbar_init(&s.pv_done[i], 1);
    }
    mbar_init(&s.o_free, 4 * G::SUMG);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.q_full[i], 4);
      mbar_init(&s.q_free[i], 5);  // the products with it, and the softmax warps' row scales
    }
    mbar_init(&s.drain, 1);
    fence_mbarrier_init();
    s.lo = 0x7fffffff;
    s.hi = 0;
    s.abort = 0;
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
  }
  if (warp == 1) tmem_alloc(&s.tmem, 512);
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  const int flags = make_plan<D>(p, s);
  const int pn = s.hi > s.lo ? (s.hi + G::KT - 1) / G::KT - s.lo / G::KT : 0;
  const long long tp = (long long)pn * p.Hkv * p.row_tiles;
  const long long total = tp + (long long)s.cum[p.B] * (p.Hkv * p.own_tiles);
  const int ctas = (int)min(total, (long long)p.grid);
  if (blockIdx.x == 0) {
    if (flags && p.dev_status) atomicOr(p.dev_status, flags);
    if (tid == 0) {
      p.ws_plan[0] = pn;
      p.ws_plan[1] = ctas;
    }
    for (int i = tid; i <= p.B; i += G::THREADS) p.ws_plan[2 + i] = s.cum[i];
  }
  long long g0 = 0, g1 = 0;
  if ((int)blockIdx.x < ctas) {
    g0 = part_start(blockIdx.x, total, ctas);
    g1 = part_start(blockIdx.x + 1, total, ctas);
  }
  if (warp < 4) {
    setmaxnreg_dec<G::REG_LOAD>();
    if (warp == 0) {
      Loader<D> ld(p, s);
      ld.run(tp, g0, g1);
      const int bad = __reduce_or_sync(0xffffffffu, ld.flags);
      if (bad && lane == 0 && p.dev_status) atomicOr(p.dev_status, bad);
      if (*(volatile int*)&s.abort) {
        // the copies in flight end before their memory is given back
        for (int r = max(0, ld.r - G::RING); r < ld.r; ++r)
          mbar_wait(&s.full[r % G::RING], (r / G::RING) & 1, nullptr, p.wait_ns);
      }
    } else if (warp == 1) {
      if (lane == 0) {
        mma_loop<D>(p, s, tp, g0, g1);
        if (*(volatile int*)&s.abort) {
          // so do the products
          mma_commit(&s.drain);
          mbar_wait(&s.drain, 0, nullptr, p.wait_ns);
        }
      }
    } else {
      q_loop<D>(p, s, tp, g0, g1);
    }
  } else if (warp < 8) {
    if constexpr (G::REG_SOFT > G::REG_LAUNCH) setmaxnreg_inc<G::REG_SOFT>();
    softmax_loop<D, CAP>(p, s, tp, g0, g1);
  } else {
    setmaxnreg_inc<G::REG_SUM>();
    sum_loop<D>(p, s, tp, g0, g1);
  }
  __syncwarp();
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  if (warp == 1) tmem_free(s.tmem, 512);
}

// ------------------------------------------------------------------ joining the states
constexpr int kMergeWarps = 8;

// One warp a row.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    prefix_merge_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const long long at = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  if (at >= (long long)p.B * p.T * p.Hq) return;
  const int row = (int)at;
  const int bt = row / p.Hq, hq = row - bt * p.Hq, h = hq / p.G;
  const int b = bt / p.T, tok = bt - b * p.T;
  const int r1 = tok * p.G + hq - h * p.G;
  const int rb = b * p.R1 + r1;
  const int pn = p.ws_plan[0], ctas = p.ws_plan[1];
  const int* cum = p.ws_plan + 2;
  const int units1 = p.Hkv * p.own_tiles;
  const long long tp = (long long)pn * p.Hkv * p.row_tiles;
  const long long total = tp + (long long)cum[p.B] * units1;
  float M = -kInf, L = 0.f, o[V];
  bool partial = false;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  auto add = [&](float2 ml, const float* src) {
    partial |= signbit(ml.y) != 0;
    if (ml.y == 0.f) return;  // no key
    const float mn = fmaxf(M, ml.x);
    const float f = ex2_ftz(M - mn), w = ex2_ftz(ml.x - mn);
    M = mn;
    L = fmaf(L, f, w * fabsf(ml.y));
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(o[i], f, w * src[lane * V + i]);
  };
  for (int u = 0; u < 2; ++u) {  // the prefix's states, then the own keys'
    long long g0;
    int n, in_tile;
    if (u == 0) {
      n = pn;
      g0 = (h * (long long)p.row_tiles + rb / kPrefixRows) * pn;
      in_tile = rb % kPrefixRows;
    } else {
      n = cum[b + 1] - cum[b];
      g0 = tp + (long long)cum[b] * units1 +
           ((long long)h * p.own_tiles + r1 / kPrefixRows) * n;
      in_tile = r1 % kPrefixRows;
    }
    if (n == 0) continue;
    const int c0 = part_cta(g0, total, ctas), c1 = part_cta(g0 + n - 1, total, ctas);
    if (c0 == c1) {
      if (u == 0)
        add(p.ws_pre_ml[row], p.ws_pre_o + (long long)row * D);
      else
        add(p.ws_own_ml[row], p.out + (long long)row * D);
      continue;
    }
    for (int c = c0; c <= c1; ++c) {
      const int slot = 2 * c + (c == c0 && part_start(c, total, ctas) != g0 ? 1 : 0);
      const long long i = (long long)slot * kPrefixRows + in_tile;
      add(p.ws_cut_ml[i], p.ws_cut_o + i * D);
    }
  }
  // A zero weight does not silence a value that is not finite: a row that met masked keys
  // and came out non-finite is done again, key by key.
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) bad |= !isfinite(o[i]);
  if (__any_sync(0xffffffffu, partial && bad)) {
    int len, qp, lo, hi;
    seq_info(p, b, len, qp);
    key_range(p, len, qp, tok, tok, lo, hi);
    float q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = p.q[(long long)row * D + lane * V + i];
    attend_row<D>(p, b, h, q, lo, hi, M, L, o);
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int i = 0; i < V; ++i) p.out[(long long)row * D + lane * V + i] = o[i] * inv;
  if (lane == 0 && p.lse) p.lse[row] = L == 0.f ? -kInf : (M + log2f(L)) * kLn2;
}

template <int D, bool CAP>
cudaError_t launch_prefix_impl(const PrefixParams& p, cudaStream_t stream) {
  constexpr int smem = (int)sizeof(PrefixSmem<D>);
  static std::atomic<int> configured[128];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 128 || !configured[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(prefix_attn_kernel<D, CAP>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 128) configured[dev].store(1, std::memory_order_release);
  }
  const long long rows = (long long)p.B * p.T * p.Hq;
  const long long blocks = (rows + kMergeWarps - 1) / kMergeWarps;
  prefix_attn_kernel<D, CAP><<<p.grid, PGeo<D>::THREADS, smem, stream>>>(p);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  prefix_merge_kernel<D><<<(int)blocks, kMergeWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, cudaStream_t stream) {
  const bool cap = p.softcap2 > 0.f;
  if (p.D == 64)
    return cap ? launch_prefix_impl<64, true>(p, stream) : launch_prefix_impl<64, false>(p, stream);
  if (p.D == 128)
    return cap ? launch_prefix_impl<128, true>(p, stream) : launch_prefix_impl<128, false>(p, stream);
  return cap ? launch_prefix_impl<256, true>(p, stream) : launch_prefix_impl<256, false>(p, stream);
}

}  // namespace da
