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
// of 64 (128 for D = 64).  A prefix unit is a (kv head, tile of the batch's
// rows) over the prefix, an own unit a (sequence, kv head, tile of its rows)
// over its own keys.  A unit's key tiles, and entries that stand for its fixed cost, form a run of
// a list; every CTA takes an equal share of entries (tiles cost about the same: the MMA's M is 128
// whether a tile has 4 rows or 128).  A unit that lies in one CTA leaves its state in
// the row's place; the parts of a unit that CTA boundaries cut go to the
// CTAs' slots.  prefix_merge_kernel joins a row's states:
// M = max m_s, w_s = 2^(m_s - M), out = sum w_s o_s / sum w_s l_s.
//
// A tile.  S = Q K^T and O_tile = P V run on the tensor cores (tcgen05), f16
// operands and f32 accumulators in tensor memory.  Q (f32) is held as
// two f16 terms of q / 2^e, e the row's exponent, P as two f16 terms of the weight times 2^8: 22 bits
// each, so out keeps f32's accuracy (one term would leave 2^-12).  Weights below 2^-22 of the
// part's largest lose bits, each off by up to 2^-33 of that: as much as an f32 sum that holds the
// largest drops of them (2^-25 of it a step), n 2^-33 of the result for n equal ones below one
// largest.  The two terms double
// the products: 8 * 128 * D flops a key; a 64-key tile of D = 128 is 1024
// cycles of the tensor pipe for 32 KB of K and V, about the rate at which
// HBM delivers them.  The tensor cores' f32 sums truncate: a long chain of
// them drifts (2^-24 of the sum a step on average; 3.6e-5 of the result after 145 tiles
// in one accumulator).  So every second tile starts a new accumulator, the low terms go first
// (their steps truncate at their own size), and the sums over tiles are ordinary f32 adds in
// registers.
//
// Warps.  0: TMA of K pages into a ring of tiles, 3: of V pages (D = 256: 0
// both, 3 the Q of units with few rows).  1 issues the scores' products, 2
// the values' (S and P share three or four buffers, so scores run
// ahead while the softmax of a tile runs).  Then two warpgroups (D = 256: one) of softmax, a
// thread a row: scores to weights, running maximum and sum; they take turns at the tiles and hand
// the maximum on, and convert Q.  Then one (D = 256: two, 128 columns each) of sums, a thread a
// row: acc = acc * 2^(m_old - m_new) + O, and the state's store.  A unit of few rows lies in the
// lanes of one warp of each of these groups, and four such units run at once.
//
// Measured (GB300), 128 sequences x 64 heads, 8 kv heads, D = 128, 32,768 shared and 64 to 2048 own
// keys: 245 to 272 us by the card, 235 of them in prefix_attn_kernel, which issues 352 GFLOP of products (140 before
// the second terms and the empty rows of own tiles): 1.5 PFLOP/s, 79% of the tensor cores' measured
// rate, at the card's power limit; 452 MB read, 1.9 TB/s.  A tile takes 0.8 us for 0.55 of products:
// the softmax's and the sums' traffic with tensor memory; an own unit's chain of latencies 2 to 3 us.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "../../include/decode_attn.h"
#include "launch.h"
#include "ptx.cuh"
#include "tc5.cuh"

namespace da {

namespace {

constexpr float kInf = INFINITY;
constexpr int kPlanInts = sizeof(PrefixPlan) / 4;
constexpr float kLn2 = 0.6931471805599453f;

// cap * tanh(y) in base-2 units.  Below |y| = 1/2 as z + z t P(t), z = cap y, t = y^2, P of degree 3
// fitted (weighted least squares until its error was level) to (tanh(y) / y - 1) / y^2: off by 1.5e-8 of
// tanh, with its roundings by 2.2 of 2^-24, relative, so a score keeps f32's accuracy whatever
// the cap.  (tanh's series needs y^13 for that, two more products: 382 us against 353 for 128 sequences of 64 heads over
// 32,768 shared keys.)  Above, by
// the identity in 2^x, whose rounding next to 1 costs 3e-7 of a tanh that is near 1: 1.5e-5 of a
// score at a cap of 50, as in the unshared kernels.  Where one score of 16 columns is past 1/2 both
// forms are worked out: 32,768 shared keys with a cap of 30 take 377 us for scores near 1, 389 and
// 511 for a spread of 4 and 8.
__device__ __forceinline__ float2 cap_near(float2 y, float cap2) {
  auto two = [](float c) { return make_float2(c, c); };
  const float2 t = mul2(y, y), z = mul2(y, two(cap2));
  float2 p = fma2(two(0.017241476f), t, two(-0.053045485f));
  p = fma2(p, t, two(0.13325879f));
  p = fma2(p, t, two(-0.33333144f));
  return fma2(z, mul2(t, p), z);
}
__device__ __forceinline__ float cap_any(float y, float cap2) {
  const float small = cap_near(make_float2(y, y), cap2).x;
  const float big = cap2 * (1.f - __fdividef(2.f, ex2_ftz(y * 2.8853900817779268f) + 1.f));
  return fabsf(y) <= 0.5f ? small : big;
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
// lower bound, token t1's upper bound.  qp is at least -T, and only then negative;
// otherwise the sums fit in 32 unsigned bits.
__device__ __forceinline__ void key_range(const PrefixParams& p, int len, int qp, int t0, int t1,
                                          int& lo, int& hi) {
  const uint32_t a = (uint32_t)qp + t0, z = (uint32_t)qp + t1 + 1;
  const bool before = qp < 0 && (int)a < 0, none = qp < 0 && (int)z <= 0;
  const uint32_t W = p.window;
  const uint32_t l = (W > 0 && !before && a >= W) ? a - W + 1 : 0;
  const uint32_t h = !p.causal ? len : none ? 0 : min(z, (uint32_t)len);
  const bool some = h > l;
  lo = some ? (int)l : 0;
  hi = some ? (int)h : 0;
}

// Page of key k of sequence b (not checked against num_blocks).
__device__ __forceinline__ int page_of(const PrefixParams& p, int b, int k) {
  const int c = k >> p.log2_bs;
  return c < p.prefix_pages ? p.prefix_table[c]
                            : p.block_table[(long long)b * p.max_blocks + c];
}

// One warp's state of a row over keys [k0, k1), four keys a step: lane i holds the values
// [i * D/32, (i + 1) * D/32) of q and o.  Pages outside the pool are masked: neither their keys nor
// their values count.  Ends early where the sum is NaN (a query that is not finite, a NaN key):
// nothing behind changes the row any more.
template <int D>
__device__ __noinline__ void attend_row(const PrefixParams& p, int b, int kv, const float (&q)[D / 32], int k0,
                           int k1, float& m, float& l, float (&o)[D / 32]) {
  constexpr int V = D / 32, N = 4;
  const int lane = threadIdx.x & 31;
  m = -kInf;
  l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
#pragma unroll 1
  for (int k = k0; k < k1 && !isnan(l); k += N) {
    long long at[N];
    bool ok[N];
    float s[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int key = min(k + u, k1 - 1), blk = page_of(p, b, key);
      ok[u] = k + u < k1 && (uint32_t)blk < (uint32_t)p.num_blocks;
      at[u] = ((((long long)(ok[u] ? blk : 0) << p.log2_bs) + (key & (p.bs - 1))) * p.Hkv + kv) * D +
              lane * V;
      s[u] = 0.f;
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(p.k_pool + at[u] + i));
        s[u] = fmaf(q[i], x.x, fmaf(q[i + 1], x.y, s[u]));
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < N; ++u) {
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], off);
      s[u] *= p.qscale;
      if (p.softcap2 > 0.f) s[u] = cap_any(s[u] * p.softcap_inv, p.softcap2);
      if (!ok[u]) s[u] = -kInf;
      mn = fmaxf(mn, s[u]);
    }
    const float base = mn == -kInf ? 0.f : mn;
    const float f = exp2f(m - base);
    l *= f;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] *= f;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const float w = exp2f(s[u] - base);
      l += w;
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(p.v_pool + at[u] + i));
        o[i] = ok[u] ? fmaf(w, x.x, o[i]) : o[i];
        o[i + 1] = ok[u] ? fmaf(w, x.y, o[i + 1]) : o[i + 1];
      }
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
  static constexpr int NS = D == 128 ? 4 : 3;     // S / P buffers
  // Tensor-memory columns: O, then (D < 256) the two terms of Q, then S / P, then, if any are
  // left, the factors.  With Q there the score products read only K from shared memory (with both
  // operands in it they ran at two thirds of their rate), and 64 KB more of it hold tiles in
  // flight.  D = 256 has no room for Q beside O.
  static constexpr bool QT = D < 256;
  static constexpr int Q0 = QT ? D : 0;
  static constexpr int S0 = Q0 + D;
  static constexpr int F0 = S0 + NS * KT;
  static constexpr bool FAC_TMEM = F0 + NS <= 512;
  // Tiles in flight: with Q in tensor memory K and V have a ring and a loading
  // warp each; else three tiles are shared, in the products' order.
  static constexpr int RK = QT ? 7 : 3, RV = QT ? 6 : 0, RING = RK + RV;
  static constexpr int AC = D < 128 ? D : 128;    // columns a sum thread holds
  static constexpr int SUMG = D / AC;             // sum warpgroups
  static constexpr int SOFTG = D >= 256 ? 1 : 2;  // softmax warpgroups, taking turns at the tiles
  static constexpr int SETS = QT ? 5 : 1;         // of barriers, by which warps take a part
  static constexpr int GROUPS = 1 + SOFTG + SUMG;
  static constexpr int THREADS = 128 * GROUPS;
  // Registers a thread: at launch, then by role (setmaxnreg); the roles'
  // sum over the warpgroups stays within the launch's.
  static constexpr int REG_LAUNCH = 128;
  static constexpr int REG_LOAD = 64;
  static constexpr int REG_SOFT = SOFTG == 1 ? 112 : 136;
  static constexpr int REG_SUM = SOFTG == 1 ? 168 : 176;
  static_assert(F0 <= 512, "tensor memory");
  static_assert(REG_LOAD + SOFTG * REG_SOFT + SUMG * REG_SUM <= GROUPS * REG_LAUNCH, "registers");
  static_assert(THREADS * REG_LAUNCH <= 65536, "registers");
};

// Parts of at most this many rows leave room for the next part's Q: a quarter of the lanes
// each in tensor memory, half of the buffer in shared memory.
template <int D>
constexpr int kSmallRows = PGeo<D>::QT ? 32 : 64;
// Units cost more than their tiles: Q, the first tile's latencies, the state's store.  The list
// counts so many tiles for it.  D = 128, 32 to 64 heads and 64 to 2048 own keys, without it (0, 0) and
// with (8, 1): 376 and 250 us over 32,768 shared keys, 61 and 43 over 8192, 419 and 78 over 16.  From
// there it is flat: (14, 1) took 252, 44, 79, (16, 2) 252, 44, 81.  D = 256: 170 without and 136 us
// with it for 64 sequences of 16 heads, a window of 4096 and 256 to 2048 own keys (nearly all of its
// tiles are own ones of two rows; full tiles of D = 256, and D = 64, were not fitted by themselves).
template <int D>
constexpr int kPrefixExtra = D >= 256 ? 20 : 8;
constexpr int kOwnExtra = 1;
// And so does a CTA's run of the prefix, wherever in a unit it begins: it decides how many CTAs the
// prefix gets.  0 and these: 134 and 114 us for the D = 256 case, 42 and 41 over 8192 shared keys,
// 27.2 and 26.2 for 32 sequences over 4096.
template <int D>
constexpr int kPartExtra = D >= 256 ? 14 : 4;
// The maximum that a tile's weights are taken against moves at the first tile of a group of
// kGroup, whose products add up in tensor memory before the sum warps take them, and where a row
// outgrows it by 2^kGrow (that tile then starts a group).  Weights are kept times 2^kShift:
// those down to 2^-22 of the largest stay normal f16 numbers, and none passes 2^15.
// (Groups of 4 and of 8 take 1 and 2% less time, 249, 247 and 245 us for the long case above, with
// twice and four times the truncating steps in a chain.)
constexpr int kGroup = 2;
constexpr float kGrow = 7.f;
constexpr float kShift = 8.f;

// A part of a unit (Part) as the CTA's run names it.
struct alignas(16) PartInfo {
  int b, h;              // b < 0: prefix
  int r0, nr;
  int base, klo, khi;    // keys [klo, khi) may be seen
  int i0, n;
  int slot;              // its rows' place among the parts of units that are cut, or -1: all of one
};
// How many a CTA keeps: a part is read by every warp before the loads are so many ahead of it (they
// are at most 13 tiles ahead of the sums, and a warp takes at least every fourth part).
constexpr int kParts = 32;

template <int D>
struct PrefixSmem {
  using G = PGeo<D>;
  static constexpr int MAXB = prefix_max_batch(D);
  uint8_t ring[G::RING * G::TILE];
  uint8_t q[G::QT ? 16 : 2 * G::QTERM];
  uint64_t full[G::RING], empty[G::RING];
  uint64_t s_full[G::SETS * G::NS], p_full[G::SETS * G::NS], pv_done[G::SETS * G::NS];
  uint64_t b_free[G::NS], o_free;
  uint64_t q_full[G::QT ? G::SETS : 2], q_free[G::QT ? G::SETS : 2], drain[2];
  uint64_t m_ready[4], l_ready[2][4], q_half[4];         // by warp of a warpgroup
  uint64_t part_ready[G::QT ? kParts : 1];
  PartInfo parts[G::QT ? kParts : 1];
  float row_scale[G::QT ? 1 : kPrefixRows];              // qscale * 2^e, by row of the Q buffer
  float fac[G::FAC_TMEM ? 1 : G::NS * kPrefixRows];      // 2^(m_old - m_new) of a tile's rows
  // two softmax warpgroups: the running maximum from one tile to the next, the sum of the one
  // that does not end the part, the largest value of their halves of a Q row
  float m[G::SOFTG == 1 ? 1 : kPrefixRows], l[G::SOFTG == 1 ? 1 : 2 * kPrefixRows],
      m_last[G::SOFTG == 1 ? 1 : 2 * kPrefixRows], q_max[G::SOFTG == 1 ? 1 : 2 * kPrefixRows];
  int cum[MAXB + 1];                                     // the list's tiles a unit before sequence b
  int len[MAXB], qp[MAXB];                               // seq_info
  int bad[16];                                           // per tile (mod 16): masked boxes of keys
  uint8_t grew[G::NS][4];                                // by tile's buffer and warp: a row outgrew
  int warp_sum[16];
  int lo, hi;                                            // prefix keys some row sees
  // the CTA's runs of the prefix's list and the own one: where they start (sequence, kv head,
  // tile of rows or block of them, entry of the unit) and how long they are
  int first[2][4], run[2];
  PrefixPlan plan;
  unsigned long long best;                               // cost and number of groups
  int skip;                                              // test hook: the first copy is left out
  int abort;
  uint32_t tmem;
};
static_assert(sizeof(PrefixSmem<64>) <= kSmemLimit && sizeof(PrefixSmem<128>) <= kSmemLimit &&
                  sizeof(PrefixSmem<256>) <= kSmemLimit,
              "shared memory");

// A list of tiles (fewer than 2^31: the host refuses more) is cut into runs
// of share + 1 tiles (the first rem CTAs) and share.
struct Split {
  int share, rem;
  __device__ __forceinline__ Split(int share_, int rem_) : share(share_), rem(rem_) {}
  __device__ __forceinline__ static Split of(int total, int ctas) {
    const int share = (uint32_t)total / (uint32_t)ctas;
    return {share, total - share * ctas};
  }
  __device__ __forceinline__ int longest() const { return share + (rem > 0); }
  __device__ __forceinline__ int start(int c) const { return c * share + min(c, rem); }
  // The CTA whose run holds tile g.
  __device__ __forceinline__ int cta(int g) const {
    const int longer = rem * (share + 1);
    return g < longer ? (uint32_t)g / (uint32_t)(share + 1)
                      : rem + (uint32_t)(g - longer) / (uint32_t)share;
  }
};

// Waits for the phase of `bar` with the given parity.  A wait that runs past
// the limit sets the abort flag; every role then leaves its loop, and the kernel reports it
// at its end.  Short, because it is inlined at every wait: the kernel's code has to stay in the
// instruction cache (123 KB of it, most in these waits, took 566 us where 61 KB took 322: 128
// sequences of 64 heads over 32,768 shared keys).
template <int D>
__device__ __forceinline__ bool wait_or_abort(const PrefixParams& p, PrefixSmem<D>& s,
                                              uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*(volatile int*)&s.abort) return false;
    if (globaltimer_ns() - t0 > p.wait_ns) {
      *(volatile int*)&s.abort = 1;
      return false;
    }
  }
  return true;
}
// The same for all lanes of a warp, which go on or leave together.
template <int D>
__device__ __forceinline__ bool warp_wait(const PrefixParams& p, PrefixSmem<D>& s, uint64_t* bar,
                                          uint32_t parity) {
  return __all_sync(0xffffffffu, wait_or_abort<D>(p, s, bar, parity));
}

// A part of a unit: rows [r0, r0 + nr) of kv head h (r0 counts the batch's rows in the prefix,
// the sequence's in its own keys), key tiles [i0, i0 + n), tile i's keys starting at base + i * KT.
template <int D>
struct Part : PartInfo {
  using G = PGeo<D>;
  int k = -1;            // number of the part
  __device__ __forceinline__ bool whole() const { return slot < 0; }
  __device__ __forceinline__ bool small() const { return nr <= kSmallRows<D>; }
  // Q in tensor memory: the rows of a small part lie in the lanes of one warp of each warpgroup,
  // and only these warps take part in it, so that four such parts are under way at once.  Barriers
  // that not every warp waits for come in sets, one of each of those warps' and one of all's (a
  // warp then waits for every phase of the barriers it knows).
  __device__ __forceinline__ bool apart() const { return G::QT && small(); }
  __device__ __forceinline__ int set() const { return apart() ? k % 4 : G::SETS - 1; }
  __device__ __forceinline__ bool takes(int w) const { return !apart() || k % 4 == w; }
  // Lane of tensor memory (row of the Q buffer) of the part's first row.
  __device__ __forceinline__ int lane0() const {
    constexpr int parts = kPrefixRows / kSmallRows<D>;
    return small() ? k % parts * kSmallRows<D> : 0;
  }
  // Sequence, query token and place in [B, T, Hq] of the part's row i.
  __device__ __forceinline__ int out_row(const PrefixParams& p, int i, int& seq, int& tok) const {
    int r = r0 + i;
    seq = b;
    if (b < 0) {
      seq = (uint32_t)r / (uint32_t)p.R1;
      r -= seq * p.R1;
    }
    tok = (uint32_t)r / (uint32_t)p.G;
    return (seq * p.T + tok) * p.Hq + h * p.G + (r - tok * p.G);
  }
};

// The parts that a CTA's runs are made of, one after the other, the prefix's first.  A unit's first
// `extra` entries of its list stand for its fixed cost; runs that hold only such entries of a unit have
// no part of it.  TELL: each is announced to the warps that read them with a Reader.
template <int D, bool TELL>
struct Lister : Part<D> {
  using Part<D>::b, Part<D>::h, Part<D>::r0, Part<D>::nr, Part<D>::base, Part<D>::klo,
      Part<D>::khi, Part<D>::i0, Part<D>::n, Part<D>::slot, Part<D>::k;
  static constexpr int KT = PGeo<D>::KT;
  const PrefixParams& p;
  PrefixSmem<D>& s;
  int left;              // entries of the run from this part on
  int at, len;           // the part's first entry of its unit, its entries
  int rt;                // tile of rows; prefix: block of them
  int moved;             // the run's first unit is behind

  __device__ __forceinline__ Lister(const PrefixParams& p_, PrefixSmem<D>& s_) : p(p_), s(s_) {
    enter(0);
    n = 0;
  }
  __device__ __forceinline__ void enter(int list) {
    b = s.first[list][0];
    h = s.first[list][1];
    rt = s.first[list][2];
    at = s.first[list][3];
    left = s.run[list];
    len = -1;
    moved = 0;
  }
  // On to the first or next part; false, and n = 0, behind the last one.
  __device__ __forceinline__ bool step() {
    if (k >= 0 && n == 0) return false;
    n = 0;
    do {
      if (len >= 0) {
        left -= len;
        at = 0;
        moved = 1;
        if (left > 0 && ++rt == (b < 0 ? s.plan.blocks : p.own_tiles)) {
          rt = 0;
          if (++h == p.Hkv) {
            h = 0;
            if (b >= 0) {
              ++b;
              while (s.cum[b + 1] == s.cum[b]) ++b;
            }
          }
        }
      }
      if (left <= 0 && b < 0) enter(1);
      if (left <= 0) break;
      int extra = kOwnExtra, unit_n, rows = p.R1;
      slot = (blockIdx.x * 2 + moved) * p.own_rows + p.grid * (2 * kPrefixRows);
      r0 = rt * kPrefixRows;
      if (b < 0) {
        extra = kPrefixExtra<D>;
        rows = p.B * p.R1;
        r0 = (rt * s.plan.width + (int)blockIdx.x % s.plan.width) * kPrefixRows;
        slot = (blockIdx.x * 2 + moved) * kPrefixRows;
        klo = s.lo;
        khi = s.hi;
        base = klo / KT * KT;
        unit_n = (khi + KT - 1) / KT - klo / KT;
      } else {
        const int P = p.prefix_pages << p.log2_bs;
        key_range(p, s.len[b], s.qp[b], 0, p.T - 1, klo, khi);
        klo = max(klo, P);
        base = P + (klo - P) / KT * KT;
        unit_n = s.cum[b + 1] - s.cum[b] - extra;
      }
      len = min(unit_n + extra - at, left);
      i0 = max(0, at - extra);
      nr = min(kPrefixRows, rows - r0);
      n = nr > 0 ? at + len - extra - i0 : 0;  // the last block may have fewer tiles
      if (n == unit_n) slot = -1;
    } while (n <= 0);
    n = max(n, 0);
    ++k;
    if (TELL && (threadIdx.x & 31) == 0) {
      s.parts[k % kParts] = *this;
      mbar_arrive(&s.part_ready[k % kParts]);
    }
    return n > 0;
  }
};

template <int D>
struct Reader : Part<D> {
  using Part<D>::k, Part<D>::n;
  const PrefixParams& p;
  PrefixSmem<D>& s;
  __device__ __forceinline__ Reader(const PrefixParams& p_, PrefixSmem<D>& s_) : p(p_), s(s_) {}
  __device__ __forceinline__ bool step() {
    const int next = k + 1, at = next % kParts;
    if (!warp_wait<D>(p, s, &s.part_ready[at], next / kParts & 1)) return false;
    static_cast<PartInfo&>(*this) = s.parts[at];
    k = next;
    return n > 0;
  }
};

// How a warp other than the one that loads K walks its CTA's parts: to find one takes 1000 cycles, as
// much as a tile, to read it 100; D = 256, whose parts are longer, has no room to keep them.
template <int D>
using Cursor = std::conditional_t<PGeo<D>::QT, Reader<D>, Lister<D, false>>;

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
    if (hi > l) n = (hi - P + KT - 1) / KT - (l - P) / KT + kOwnExtra;
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

// Shares the work out: runs of equal length, the prefix's entries and the own ones together.
// CTAs that work on the same keys for different tiles of rows should do so at the same
// time, or each reads them from HBM: `width` neighbours form a group that goes through a
// list of (kv head, block of `width` tiles of rows) together, a tile of rows each.  The widest
// groups are taken that cost no more than 1/24 in balance (they leave places of the last block
// empty and grid % width CTAs out).  The CTAs behind the groups take the own list, the groups' what
// is left of it.  128 sequences of 64 heads, 8 tiles of rows, over 32,768 shared keys: single
// CTAs read 787 MB of HBM in 235 us, groups 151 in 203; with 64 to 2048 own keys besides 862 MB and 262
// us, 452 and 252.
// All threads call it, one a width.
template <int D>
__device__ void share_out(const PrefixParams& p, PrefixSmem<D>& s) {
  const int tid = threadIdx.x;
  const int pn = s.hi > s.lo ? (s.hi + PGeo<D>::KT - 1) / PGeo<D>::KT - s.lo / PGeo<D>::KT +
                                   kPrefixExtra<D>
                             : 0;
  const int units1 = p.Hkv * p.own_tiles, own = s.cum[p.B] * units1;
  // entries of a run where tiles of rows are worked on `width` at a time
  auto mean = [&](int width, int blocks) {
    return (int)(((uint32_t)pn * (p.Hkv * blocks) * width + own + p.grid - 1) / (uint32_t)p.grid);
  };
  if (p.row_tiles > 1 && tid < (pn ? min(p.row_tiles, p.grid) : 0)) {
    const int width = tid + 1, blocks = (uint32_t)(p.row_tiles + tid) / (uint32_t)width;
    const Split pre = Split::of(pn * (p.Hkv * blocks), (uint32_t)p.grid / (uint32_t)width);
    const int longest = max(pre.longest(), mean(width, blocks));
    if ((long long)longest * 24 <= (long long)mean(1, p.row_tiles) * 25)
      atomicMax(&s.plan.width, width);
  }
  __syncthreads();
  const int c = blockIdx.x, width = s.plan.width;
  const int blocks = (uint32_t)(p.row_tiles + width - 1) / (uint32_t)width;
  const int tp = pn * (p.Hkv * blocks);
  // How many groups: a run of the prefix costs its CTA kPartExtra more than its entries (Q of 128 rows,
  // their state), whatever unit it is of.  One thread a number.
  const int most = min((uint32_t)p.grid / (uint32_t)width, (uint32_t)(p.Hkv * blocks * 32));
  if (tid < (pn ? most : 0)) {
    const int n = tid + 1;
    const uint32_t all =
        (uint32_t)tp * width + (uint32_t)(n * width * kPartExtra<D>) + own + p.grid - 1;
    const int cost = max(Split::of(tp, n).longest() + kPartExtra<D>, (int)(all / (uint32_t)p.grid));
    atomicMin(&s.best, (unsigned long long)cost << 32 | (unsigned)n);
  }
  __syncthreads();
  if (tid != 0 && tid != 32) return;
  const int groups = pn ? (int)(uint32_t)s.best : p.grid;
  const int each = pn ? (int)(s.best >> 32) : mean(1, 1);
  const Split pre = Split::of(tp, groups);
  const int members = groups * width, others = p.grid - members;
  // all own entries where that fits (a few for each member would cut units for little)
  const int room = others * each, before = (long long)own * 24 <= (long long)room * 25 ? own : room;
  const Split front = Split::of(before, max(others, 1)), rest = Split::of(own - before, members);
  if (tid == 0) {
    s.plan = {pn,     width,  blocks,      pre.share, pre.rem,    members,
              others, before, front.share, front.rem, rest.share, rest.rem};
    const int group = (uint32_t)c / (uint32_t)width, g = pre.start(group);
    s.run[0] = group < groups ? pre.share + (group < pre.rem) : 0;
    s.first[0][0] = -1;
    if (s.run[0] > 0) {
      const int u = (uint32_t)g / (uint32_t)pn;
      s.first[0][1] = (uint32_t)u / (uint32_t)blocks;
      s.first[0][2] = u - s.first[0][1] * blocks;
      s.first[0][3] = g - u * pn;
    }
    // test hook: the first tile of the first CTA that has one
    if (pn > 0)
      s.skip = p.test_skip_arm && c == group * width && g <= kPrefixExtra<D> &&
               kPrefixExtra<D> < g + s.run[0];
    return;
  }
  const int o = c < members ? c : c - members;
  int g = c < members ? before + rest.start(o) : front.start(o);
  s.run[1] = c < members ? rest.share + (o < rest.rem) : front.share + (o < front.rem);
  if (pn == 0) s.skip = p.test_skip_arm && g <= kOwnExtra && kOwnExtra < g + s.run[1];
  if (s.run[1] > 0) {
    const int x = (uint32_t)g / (uint32_t)units1;  // sequence b holds it: cum[b] <= x < cum[b + 1]
    int b = 0, hi = p.B;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (s.cum[mid] <= x)
        b = mid;
      else
        hi = mid;
    }
    g -= s.cum[b] * units1;
    const int u = (uint32_t)g / (uint32_t)(s.cum[b + 1] - s.cum[b]);
    s.first[1][0] = b;
    s.first[1][1] = (uint32_t)u / (uint32_t)p.own_tiles;
    s.first[1][2] = u - s.first[1][1] * p.own_tiles;
    s.first[1][3] = g - u * (s.cum[b + 1] - s.cum[b]);
  }
}

// Parity of the phases of a tile's barriers (by set and buffer) as one warp comes to them: with
// one set it follows from the tile's number, else each barrier's uses so far are counted.
template <int D>
struct Phases {
  uint32_t odd = 0;
  // of barrier `at`'s next use, for tile x
  __device__ __forceinline__ uint32_t next(int at, int x) {
    if constexpr (PGeo<D>::SETS == 1) return x / PGeo<D>::NS & 1;
    const uint32_t parity = odd >> at & 1;
    odd ^= 1u << at;
    return parity;
  }
  // of its last use, for tile x
  __device__ __forceinline__ uint32_t last(int at, int x) const {
    if constexpr (PGeo<D>::SETS == 1) return x / PGeo<D>::NS & 1;
    return odd >> at & 1 ^ 1;
  }
};

// ------------------------------------------------------------------ the ring
// The shared ring (D = 256) takes K and V in the products' order K(0) K(1) V(0) K(2) V(1) ...:
// slot of tile x's, and how often the slot was used before.
template <int D>
struct Place {
  int slot, use;
  __device__ __forceinline__ explicit Place(int at)
      : slot(at % PGeo<D>::RING), use(at / PGeo<D>::RING) {}
  __device__ __forceinline__ static Place k(int x) { return Place(x < 2 ? x : 2 * x - 1); }
  __device__ __forceinline__ static Place v(int x) { return Place(2 * x + 2); }
};

// ------------------------------------------------------------------ TMA warps
// K and V tiles into the ring.  Each lane copies one box.  Boxes without a
// visible key and pages outside the pool are filled with zeros by a copy that
// starts past the pool's last row.  No copy waits for its block ids.  One warp that loads K
// or V alone has about 1000 cycles a tile (D = 128): it reads 32 ids at once, two windows ahead,
// and does little else (with the general form's cursor and divisions, 1700).
template <int D>
struct Loader {
  using G = PGeo<D>;
  struct Tile {
    int h, k0;     // kv head; first key of this lane's box
    int blk;       // its page, where a key of it may be seen
    bool seen;
    bool there;    // false behind the last tile
  };
  const PrefixParams& p;
  PrefixSmem<D>& s;
  int nsl, sub, slice, boxes;
  uint32_t used = 0;  // bit per slot: parity of its last copy, shifted by 16 if there was one
  int flags = 0;

  __device__ __forceinline__ Loader(const PrefixParams& p_, PrefixSmem<D>& s_) : p(p_), s(s_) {
    const int lane = threadIdx.x & 31;
    nsl = G::SL / p.box_slices;
    boxes = G::KT / p.box_rows * nsl;
    sub = lane / nsl;
    slice = lane - sub * nsl;
  }
  __device__ __forceinline__ bool copies() const { return (threadIdx.x & 31) < boxes; }
  // Tile j of the cursor's part, or the next part's first.
  __device__ __forceinline__ Tile fetch(Cursor<D>& c, int& j) const {
    Tile t = {0, 0, 0, false, false};
    if (j == c.n) {
      j = 0;
      if (!c.step()) return t;
    }
    t.there = true;
    t.h = c.h;
    t.k0 = c.base + (c.i0 + j) * G::KT + sub * p.box_rows;
    t.seen = copies() && t.k0 < c.khi && t.k0 + p.box_rows > c.klo;
    if (t.seen) {
      const int* table = c.b < 0 ? p.prefix_table : p.block_table + (long long)c.b * p.max_blocks;
      t.blk = table[t.k0 >> p.log2_bs];
    }
    ++j;
    return t;
  }
  // K or V of tile number x of the CTA's run.
  __device__ __forceinline__ bool issue(const Tile& t, int x, bool is_v) {
    const int lane = threadIdx.x & 31;
    const Place<D> at = is_v ? Place<D>::v(x) : Place<D>::k(x);
    if (at.use > 0 && !warp_wait<D>(p, s, &s.empty[at.slot], (at.use - 1) & 1)) return false;
    int row = p.num_blocks << p.log2_bs;
    const bool bad = t.seen && (t.blk < 0 || t.blk >= p.num_blocks);
    if (t.seen && !bad) row = (t.blk << p.log2_bs) + (t.k0 & (p.bs - 1));
    if (!is_v) {
      const int mask = __reduce_or_sync(0xffffffffu, bad ? 1 << sub : 0);
      if (lane == 0) s.bad[x & 15] = mask;
      if (bad) flags |= DEV_BAD_BLOCK;
    }
    // test hook: a tile that never arrives; its consumer's wait runs out
    const bool skip = s.skip && x == 0 && !is_v;
    if (!skip) {
      used = (used & ~(1u << at.slot)) | (uint32_t)(at.use & 1) << at.slot | 0x10000u << at.slot;
      if (lane == 0) mbar_arrive_expect_tx(&s.full[at.slot], G::TILE);
      __syncwarp();
      if (copies())
        tma_load_4d(s.ring + at.slot * G::TILE + slice * (G::KT * 128) + sub * p.box_rows * 128,
                    is_v ? &p.tm_v : &p.tm_k, &s.full[at.slot], 0, row, slice, t.h);
    }
    return true;
  }
  // K or V into a ring of its own: slots [first, first + ring).
  template <int RING, class Parts>
  __device__ __forceinline__ void run_one(bool is_v, int first) {
    const int lane = threadIdx.x & 31;
    const bool copy = copies();
    const int none = p.num_blocks << p.log2_bs, mask = p.bs - 1;
    const CUtensorMap* map = is_v ? &p.tm_v : &p.tm_k;
    uint8_t* to = s.ring + first * G::TILE + slice * (G::KT * 128) + sub * p.box_rows * 128;
    int slot = 0, x = 0;
    uint32_t parity = 1;  // of the slot's last release: none to wait for the first time round
    bool skip = s.skip && !is_v;  // test hook
    for (Parts c(p, s); c.step();) {
      const int* table = c.b < 0 ? p.prefix_table : p.block_table + (long long)c.b * p.max_blocks;
      const int end = (c.khi + mask) >> p.log2_bs;  // columns that hold a key
      int k0 = c.base + c.i0 * G::KT + sub * p.box_rows;  // this lane's box
      int w0 = (c.base + c.i0 * G::KT) >> p.log2_bs;
      auto window = [&](int w) { return w + lane < end ? table[w + lane] : -1; };
      int ids = window(w0), more = window(w0 + 32);
#pragma unroll 1
      for (int j = 0; j < c.n; ++j, ++x, k0 += G::KT) {
        const int col = (k0 >> p.log2_bs) - w0;
        const int a = __shfl_sync(0xffffffffu, ids, col), b = __shfl_sync(0xffffffffu, more, col);
        const int blk = col < 32 ? a : b;
        const bool seen = copy && k0 < c.khi && k0 + p.box_rows > c.klo;
        const bool ok = (uint32_t)blk < (uint32_t)p.num_blocks;
        const int row = seen && ok ? (blk << p.log2_bs) + (k0 & mask) : none;
        if (x >= RING && !warp_wait<D>(p, s, &s.empty[first + slot], parity)) return;
        if (!is_v) {
          int bad = 0;
          if (__any_sync(0xffffffffu, seen && !ok)) {
            bad = __reduce_or_sync(0xffffffffu, seen && !ok ? 1 << sub : 0);
            flags = DEV_BAD_BLOCK;
          }
          if (lane == 0) s.bad[x & 15] = bad;
        }
        if (!skip) {
          const int at = first + slot;
          used = (used & ~(1u << at)) | (parity ^ 1) << at | 0x10000u << at;
          if (lane == 0) mbar_arrive_expect_tx(&s.full[at], G::TILE);
          __syncwarp();
          if (copy) tma_load_4d(to + slot * G::TILE, map, &s.full[at], 0, row, slice, c.h);
        }
        skip = false;
        if (++slot == RING) {
          slot = 0;
          parity ^= 1;
        }
        // all boxes of the next tile lie in the second window
        if (__shfl_sync(0xffffffffu, ((k0 + G::KT) >> p.log2_bs) - w0, 0) >= 32) {
          w0 += 32;
          ids = more;
          more = window(w0 + 32);
        }
      }
    }
  }
  // One warp loads both, in the order of the shared ring.
  __device__ __forceinline__ void run_both() {
    Cursor<D> c(p, s);
    int j = 0;
    Tile t0 = {0, 0, 0, false, false}, t1 = t0, t2 = t0;  // tiles x, x + 1, x + 2
#pragma unroll 1
    for (int x = -3; x < 0 || t0.there; ++x) {
#pragma unroll 1
      for (int u = x < 0 ? 1 : 0; u < (t2.there ? 2 : 1); ++u)
        if (!issue(u ? t2 : t0, u ? x + 2 : x, u == 0)) return;
      t0 = t1;
      t1 = t2;
      t2 = fetch(c, j);
    }
  }
  // After an abort: the copies in flight end before their memory is given back.
  __device__ __forceinline__ void drain() {
    for (int i = 0; i < G::RING; ++i)
      if (used >> (16 + i) & 1) mbar_wait(&s.full[i], used >> i & 1, nullptr, p.wait_ns);
  }
};

// What a softmax thread knows of its row in a part.
struct Row {
  bool any, on;       // the warp has rows, the thread has one
  int lo, hi;         // keys it sees among the part's
  int place;          // in [B, T, Hq]; of the part's nearest row where the thread has none
  float scale;        // of its scores, base 2
  float m, l;         // running maximum, and the sum of the weights against it
};
// Its place (of sequence b, query token tok).
template <int D>
__device__ __forceinline__ int row_place(const PrefixParams& p, const Part<D>& c, int w, int& b,
                                         int& tok) {
  const int row = w * 32 + (int)(threadIdx.x & 31);
  return c.out_row(p, min(max(row - c.lane0(), 0), c.nr - 1), b, tok);
}
template <int D>
__device__ __forceinline__ Row row_of(const PrefixParams& p, const PrefixSmem<D>& s,
                                      const Part<D>& c, int w, int place, int b, int tok) {
  Row r = {false, false, 0, 0, place, 0.f, -kInf, 0.f};
  const int first = c.lane0(), row = w * 32 + (int)(threadIdx.x & 31);
  r.any = w * 32 + 32 > first && w * 32 < first + c.nr;
  r.on = row >= first && row < first + c.nr;
  if (r.on) {
    key_range(p, s.len[b], s.qp[b], tok, tok, r.lo, r.hi);
    const int P = p.prefix_pages << p.log2_bs;
    if (c.b < 0)
      r.hi = min(r.hi, P);
    else
      r.lo = max(r.lo, P);
  }
  return r;
}

// ------------------------------------------------------------------ Q
// A row of Q is divided by the power of two that brings its largest value to [2^9, 2^10) and
// held as two f16 terms.  Powers for a row whose largest value is m: what it is multiplied by,
// and what undoes it.  The exponent is kept in [-100, 127], where both are normal: below, a row's
// scores are next to nothing, above it is infinite.
__device__ __forceinline__ void q_powers(float m, float& by, float& undo) {
  int e = (int)(__float_as_uint(m) >> 23) - 127;
  e = min(max(e, -100), 127);
  by = __uint_as_float((uint32_t)(9 - e + 127) << 23);
  undo = __uint_as_float((uint32_t)(e - 9 + 127) << 23);
}

// Q in tensor memory: warp w of softmax group g converts half g of the rows of
// the part that lie in lanes [32 w, 32 w + 32), a thread a row.  The groups tell each other
// their halves' largest values; `uses` counts that.  Gives the thread's row, with qscale * 2^e.
template <int D>
__device__ __forceinline__ bool load_q_lanes(const PrefixParams& p, PrefixSmem<D>& s,
                                             const Part<D>& c, int group, int w, uint32_t lanes,
                                             int uses, Row& r) {
  constexpr int H = D / 2;
  const int lane = threadIdx.x & 31, row = w * 32 + lane;
  int seq, tok;
  const int at = row_place<D>(p, c, w, seq, tok);
  const float* src = p.q + (long long)at * D + group * H;
  // Every lane reads lines of its own, which is what the L1's rate bounds: each line once,
  // in the widest pieces the address allows (read twice in 16-byte ones, 128 rows took
  // 8000 cycles more).
  float v[H];
  if (reinterpret_cast<uintptr_t>(p.q) % 32 == 0) {
#pragma unroll
    for (int i = 0; i < H; i += 8) load_f32x8(src + i, v + i);
  } else {
#pragma unroll
    for (int i = 0; i < H; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(src + i);
      v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
    }
  }
  r = row_of<D>(p, s, c, w, at, seq, tok);  // while they are on their way
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < H; ++i) m = fmaxf(m, fabsf(v[i]));
  s.q_max[group * kPrefixRows + row] = m;
  __syncwarp();
  if (lane == 0) mbar_arrive(&s.q_half[w]);
  if (!warp_wait<D>(p, s, &s.q_half[w], uses & 1)) return false;
  float by;
  q_powers(fmaxf(m, s.q_max[(group ^ 1) * kPrefixRows + row]), by, r.scale);
  r.scale *= p.qscale;
#pragma unroll
  for (int i = 0; i < H; i += 16) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      split_half2(v[i + 2 * u] * by, v[i + 2 * u + 1] * by, hi[u], lo[u]);
    const uint32_t to = lanes + PGeo<D>::Q0 + (group * H + i) / 2;
    tmem_st8(to, hi);
    tmem_st8(to + D / 2, lo);
  }
  tmem_wait_st();
  tc5_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&s.q_full[c.set()]);
  return true;
}

// Q in shared memory: n <= 32 rows into rows row0 .. of the buffer by one warp;
// lane i names row i (`mine`, its place in [B, T, Hq]; lanes past the last name the last).
// A lane takes 8 values, D / 8 lanes a row: 16-byte stores.  All rows are touched first, so
// that the loop over them, kept small, finds them in L1.
template <int D>
__device__ __forceinline__ void load_q_rows(const float* src, float qscale, PrefixSmem<D>& s,
                                            int mine, int row0, int n) {
  constexpr int LR = D / 8;        // lanes of a row
  constexpr int RW = 32 / LR;      // rows of a step
  constexpr int LINES = D / 32;    // 128-byte lines of a row
  const int lane = threadIdx.x & 31, sub = lane / LR, d = lane % LR * 8;
#pragma unroll 1
  for (int i = 0; i < n; i += 32 / LINES) {
    const int at = __shfl_sync(0xffffffffu, mine, min(i + lane / LINES, 31));
    uint32_t unused;
    asm volatile("ld.global.b32 %0, [%1];"
                 : "=r"(unused)
                 : "l"(src + (long long)at * D + lane % LINES * 32));
  }
#pragma unroll 1
  for (int i = 0; i < n; i += RW) {
    const int at = __shfl_sync(0xffffffffu, mine, min(i + sub, 31));
    const float4* q = reinterpret_cast<const float4*>(src + (long long)at * D + d);
    const float4 x = q[0], y = q[1];
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    const int row = row0 + min(i + sub, n - 1);
    float m = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) m = fmaxf(m, fabsf(v[u]));
#pragma unroll
    for (int o = LR / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float f, undo;
    q_powers(m, f, undo);
    if (d == 0) s.row_scale[row] = qscale * undo;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) split_half2(v[2 * u] * f, v[2 * u + 1] * f, hi[u], lo[u]);
    const int to = (d >> 6) * (kPrefixRows * 128) + row * 128 + ((((d & 63) >> 3) ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(s.q + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(s.q + PGeo<D>::QTERM + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Rows [first, first + 32) of the cursor's part, as far as `last`.
template <int D>
__device__ __forceinline__ void load_q(const PrefixParams& p, PrefixSmem<D>& s,
                                       const Part<D>& c, int first, int last) {
  const int n = min(32, min(last, c.nr) - first);
  if (n <= 0) return;
  int seq, tok;
  const int mine = c.out_row(p, first + min((int)(threadIdx.x & 31), n - 1), seq, tok);
  load_q_rows<D>(p.q, p.qscale, s, mine, c.lane0() + first, n);
}

// Warp 3: Q of the parts with few rows, one part ahead of the products.  The
// softmax warps load the others; this warp waits for and passes those too: a
// barrier's parity names a phase only to a warp that no phase can leave behind.
template <int D>
__device__ void q_loop(const PrefixParams& p, PrefixSmem<D>& s) {
  const int lane = threadIdx.x & 31;
  bool prev_small = true;
  for (Cursor<D> c(p, s); c.step();) {
    const int k = c.k;
    const bool small = c.small();
    // a part of many rows takes the whole buffer, one of few the half of part k - 2
    if (k >= 2 && !warp_wait<D>(p, s, &s.q_free[k & 1], ((k - 2) >> 1) & 1)) return;
    if (k >= 1 && !(small && prev_small) &&
        !warp_wait<D>(p, s, &s.q_free[(k - 1) & 1], ((k - 1) >> 1) & 1))
      return;
    if (small) {
#pragma unroll 1
      for (int i = 0; i < c.nr; i += 32) load_q<D>(p, s, c, i, c.nr);
    }
    // its own arrival, and for few rows those of the softmax warps
    if (lane < 1 + (small ? 4 * PGeo<D>::SOFTG : 0)) mbar_arrive(&s.q_full[k & 1]);
    prev_small = small;
  }
}

// ------------------------------------------------------------------ softmax warps
// Largest of N scores, four chains.
template <int N>
__device__ __forceinline__ float largest(const float* v) {
  float mx[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) mx[i] = v[i];
#pragma unroll
  for (int i = 4; i < N; ++i) mx[i & 3] = fmaxf(mx[i & 3], v[i]);
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// N columns of this warp's lanes, a multiple of 32, waited for.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 32) tmem_ld32(addr + i, v + i);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; i += 32) tmem_loaded32(v + i);
}

// Scores of tile x (number j of the part) to weights.  Where two groups take turns the
// running maximum comes from the tile before and goes on to the next; `turn` counts the tiles
// that this warp's lanes took part in.
template <int D, bool CAP>
__device__ __forceinline__ bool softmax_tile(const PrefixParams& p, PrefixSmem<D>& s,
                                             const Part<D>& c, Row& r, int j, int x, int turn,
                                             int w, uint32_t lanes, int box_shift) {
  using G = PGeo<D>;
  constexpr int KT = G::KT;
  constexpr bool TWO = G::SOFTG == 2;
  const int buf = x % G::NS, lane = threadIdx.x & 31, row = w * 32 + lane;
  const uint32_t sa = lanes + G::S0 + buf * KT;
  const float cc = CAP ? 1.f : r.scale;
  float top = -kInf;
  if (r.any) {
    tc5_fence_after();
    const int k0 = c.base + (c.i0 + j) * KT;
    const int bad = s.bad[x & 15];
    const bool masked =
        !__all_sync(0xffffffffu, (!r.on || (r.lo <= k0 && r.hi >= k0 + KT)) && bad == 0);
    const float to_y = r.scale * p.softcap_inv;
    // Two passes over the scores, W or 32 columns a step: loops that stay in the
    // instruction cache and need few registers.
    constexpr int W = CAP ? 16 : 32;
#pragma unroll 1
    for (int i0 = 0; i0 < KT; i0 += W) {
      float v[W];
      if constexpr (CAP) {
        tmem_load16(sa + i0, v);
        float far = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          v[i] *= to_y;
          far = fmaxf(far, fabsf(v[i]));
        }
        if (__any_sync(0xffffffffu, far > 0.5f)) {
#pragma unroll
          for (int i = 0; i < W; ++i) v[i] = cap_any(v[i], p.softcap2);
        } else {  // NaN stays NaN
#pragma unroll
          for (int i = 0; i < W; i += 2) {
            const float2 y = cap_near(make_float2(v[i], v[i + 1]), p.softcap2);
            v[i] = y.x;
            v[i + 1] = y.y;
          }
        }
      } else {
        tmem_load<W>(sa + i0, v);
      }
      if (masked) {
        // bit i: key k0 + i0 + i is seen
        const int a = min(max(r.lo - k0 - i0, 0), 32), z = min(max(r.hi - k0 - i0, 0), 32);
        uint32_t seen = (uint32_t)(0xffffffffull << a) & ~(uint32_t)(0xffffffffull << z);
#pragma unroll
        for (int i = 0; i < W; i += 8)
          if ((bad >> ((i0 + i) >> box_shift)) & 1) seen &= ~(0xffu << i);
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (!(seen >> i & 1)) v[i] = -kInf;
      }
      if (CAP || masked) {
#pragma unroll
        for (int i = 0; i < W; i += 16)
          tmem_st16(sa + i0 + i, reinterpret_cast<const uint32_t*>(v + i));
      }
      top = fmaxf(top, largest<W>(v));
    }
    if (CAP || masked) tmem_wait_st();
  }
  float before = r.m;
  if (TWO) {
    if (turn > 0 && !warp_wait<D>(p, s, &s.m_ready[w], (turn - 1) & 1)) return false;
    before = j > 0 ? s.m[row] : -kInf;
  }
  const float most = fmaxf(before, top * cc);
  const bool grew = __any_sync(0xffffffffu, r.on && most > before + kGrow);
  const float now = grew || j % kGroup == 0 ? most : before;
  if (c.apart())
    *reinterpret_cast<uint32_t*>(s.grew[buf]) = grew;
  else if (lane == 0)
    s.grew[buf][w] = grew;
  if (TWO) {
    s.m[row] = now;
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.m_ready[w]);
  }
  if (r.any) {
    // no key so far: any finite reference does
    const float ref = now == -kInf ? 0.f : now;
    const float f = ex2_ftz(before - ref);  // for the sums up to the tile before
    if constexpr (G::FAC_TMEM)
      tmem_st1(lanes + G::F0 + buf, f);
    else
      s.fac[buf * kPrefixRows + row] = f;
    const float base = ref - kShift;
    const float2 cc2 = make_float2(cc, cc), base2 = make_float2(-base, -base);
    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll 1
    for (int i0 = 0; i0 < KT; i0 += 32) {
      float v[32];
      uint32_t ph[16], pl[16];
      tmem_load<32>(sa + i0, v);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float2 e = fma2(make_float2(v[i], v[i + 1]), cc2, base2);
        e.x = ex2_ftz(e.x);
        e.y = ex2_ftz(e.y);
        if (i & 2)
          sum1 = add2(sum1, e);
        else
          sum0 = add2(sum0, e);
        const __half2 hh = __floats2half2_rn(e.x, e.y);
        const float2 hf = __half22float2(hh);
        const float2 rest = add2(e, make_float2(-hf.x, -hf.y));
        const __half2 hl = __floats2half2_rn(rest.x, rest.y);
        ph[i / 2] = *reinterpret_cast<const uint32_t*>(&hh);
        pl[i / 2] = *reinterpret_cast<const uint32_t*>(&hl);
      }
      // the weights of 32 keys take the columns of their scores: 16 of high terms, 16 of low
      tmem_st16(sa + i0, ph);
      tmem_st16(sa + i0 + 16, pl);
    }
    // l counts against `now`, so far against the maximum this thread saw last
    r.l = fmaf(r.l, ex2_ftz(r.m - ref), (sum0.x + sum0.y) + (sum1.x + sum1.y));
    tmem_wait_st();
    tc5_fence_before();
  }
  r.m = now;
  __syncwarp();
  if (lane == 0) mbar_arrive(&s.p_full[c.set() * G::NS + buf]);
  return true;
}

template <int D>
__device__ __forceinline__ void store_ml(const PrefixParams& p, const Part<D>& c, const Row& r,
                                         int w) {
  if (!r.on) return;
  float2* dst;
  if (!c.whole())
    dst = p.ws_cut_ml + c.slot + w * 32 + (int)(threadIdx.x & 31) - c.lane0();
  else
    dst = (c.b < 0 ? p.ws_pre_ml : p.ws_own_ml) + r.place;
  *dst = make_float2(r.m - kShift, r.l);
}

// One group, Q in shared memory (D = 256).
template <int D, bool CAP>
__device__ void softmax_loop_one(const PrefixParams& p, PrefixSmem<D>& s) {
  using G = PGeo<D>;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const uint32_t lanes = s.tmem + ((uint32_t)(w * 32) << 16);
  const int box_shift = __ffs(p.box_rows) - 1;
  int x = 0;
  for (Cursor<D> c(p, s); c.step();) {
    const int k = c.k;
    if (!c.small()) {
      // many rows: they take the whole buffer
      if (k >= 1 && !warp_wait<D>(p, s, &s.q_free[(k - 1) & 1], ((k - 1) >> 1) & 1)) return;
      load_q<D>(p, s, c, w * 32, w * 32 + 32);
      if (lane == 0) mbar_arrive(&s.q_full[k & 1]);
    }
    int b, tok;
    const int place = row_place<D>(p, c, w, b, tok);
    Row r = row_of<D>(p, s, c, w, place, b, tok);
    for (int j = 0; j < c.n; ++j, ++x) {
      if (!warp_wait<D>(p, s, &s.s_full[x % G::NS], (x / G::NS) & 1)) return;
      if (j == 0) {
        if (r.on) r.scale = s.row_scale[w * 32 + lane];
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.q_free[k & 1]);
      }
      if (!softmax_tile<D, CAP>(p, s, c, r, j, x, x, w, lanes, box_shift)) return;
    }
    store_ml<D>(p, c, r, w);
  }
}

// Two groups that take turns at the tiles, Q in tensor memory.  Warp w of both loads its
// rows of a part's Q when the products of the part it took before are done with theirs; the two
// meet there, so that neither is a part ahead of the other.
template <int D, bool CAP>
__device__ void softmax_loop_two(const PrefixParams& p, PrefixSmem<D>& s) {
  using G = PGeo<D>;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const int group = (threadIdx.x >> 7) - 1;  // takes the tiles x = group mod 2
  const int row = w * 32 + lane;
  const uint32_t lanes = s.tmem + ((uint32_t)(w * 32) << 16);
  const int box_shift = __ffs(p.box_rows) - 1;
  int x = 0;                    // tiles so far, of all parts
  int turn = 0;                 // of this warp's parts
  int taken = 0;                // its parts
  int shared_sums[2] = {0, 0};  // those, by parity, whose sum took both groups
  Phases<D> phases;             // of s_full
  uint32_t q_odd = 0;           // by set: parity of the releases waited for
  int before = 0;               // the set of this warp's last part
  for (Cursor<D> c(p, s); c.step();) {
    if (!c.takes(w)) {
      x += c.n;
      continue;
    }
    const int set = c.set();
    if (taken > 0) {
      if (!warp_wait<D>(p, s, &s.q_free[before], q_odd >> before & 1)) return;
      q_odd ^= 1u << before;
    }
    before = set;
    Row r;
    if (!load_q_lanes<D>(p, s, c, group, w, lanes, taken, r)) return;
    for (int j = 0; j < c.n; ++j, ++x, ++turn) {
      const int at = set * G::NS + x % G::NS;
      const uint32_t parity = phases.next(at, x);
      if ((x & 1) != group) continue;
      if (!warp_wait<D>(p, s, &s.s_full[at], parity)) return;
      if (!softmax_tile<D, CAP>(p, s, c, r, j, x, turn, w, lanes, box_shift)) return;
    }
    const int q = taken++ & 1;
    const bool last = ((x - 1) & 1) == group;
    if (c.n > 1) {
      // the group of the part's last tile adds the other's sum to its own
      float* slot = s.l + q * kPrefixRows + row;
      if (!last) {
        *slot = r.l;
        s.m_last[q * kPrefixRows + row] = r.m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.l_ready[q][w]);
        ++shared_sums[q];
        continue;
      }
      if (!warp_wait<D>(p, s, &s.l_ready[q][w], shared_sums[q] & 1)) return;
      ++shared_sums[q];
      const float lx = *slot, mx = s.m_last[q * kPrefixRows + row];
      r.l = fmaf(lx, ex2_ftz(mx - (r.m == -kInf ? 0.f : r.m)), r.l);
    } else if (!last) {
      continue;  // the one tile was the other group's
    }
    store_ml<D>(p, c, r, w);
  }
}

// ------------------------------------------------------------------ sum warps
template <int D>
__device__ void sum_loop(const PrefixParams& p, PrefixSmem<D>& s) {
  using G = PGeo<D>;
  constexpr int C = G::AC;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const int row = w * 32 + lane, col = ((int)(threadIdx.x >> 7) - 1 - G::SOFTG) * C;
  const uint32_t lanes = s.tmem + ((uint32_t)(w * 32) << 16);
  int x = 0;
  Phases<D> phases;  // of p_full and pv_done
  for (Cursor<D> c(p, s); c.step();) {
    if (!c.takes(w)) {
      x += c.n;
      continue;
    }
    const int set = c.set() * G::NS, arrivals = c.apart() ? 4 : 1;
    const int first = c.lane0();
    const bool any = w * 32 + 32 > first && w * 32 < first + c.nr;
    const bool on = row >= first && row < first + c.nr;
    float2 acc[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) acc[i] = make_float2(0.f, 0.f);
    float fac = 0.f;  // the group's
    for (int j = 0; j <= c.n; ++j) {
      bool start = true;  // of a group, or the part's end
      float f = 0.f;
      if (j < c.n) {
        const int buf = x % G::NS;
        if (!warp_wait<D>(p, s, &s.p_full[set + buf], phases.next(set + buf, x))) return;
        start = j % kGroup == 0 || *reinterpret_cast<const uint32_t*>(s.grew[buf]) != 0;
        if (any) {
          if constexpr (G::FAC_TMEM) {
            tc5_fence_after();
            f = tmem_ld1(lanes + G::F0 + buf);
            tc5_fence_before();
          } else {
            f = s.fac[buf * kPrefixRows + row];
          }
        }
        __syncwarp();
        if (lane < arrivals) mbar_arrive(&s.b_free[buf]);
        ++x;
      }
      if (!start) continue;
      if (j > 0) {
        // the group before: its last tile is number y
        const int y = j < c.n ? x - 2 : x - 1, at = set + y % G::NS;
        if (!warp_wait<D>(p, s, &s.pv_done[at], phases.last(at, y))) return;
        if (any) {
          tc5_fence_after();
          const float2 f2 = make_float2(fac, fac);
#pragma unroll
          for (int i = 0; i < C; i += 16) {
            float o[16];
            tmem_load16(lanes + col + i, o);
#pragma unroll
            for (int u = 0; u < 16; u += 2)
              acc[(i + u) / 2] = fma2(acc[(i + u) / 2], f2, make_float2(o[u], o[u + 1]));
          }
          tc5_fence_before();
        }
        __syncwarp();
        if (lane < arrivals) mbar_arrive(&s.o_free);
      }
      fac = f;
    }
    if (on) {
      float* dst;
      if (!c.whole()) {
        dst = p.ws_cut_o + (long long)(c.slot + row - first) * D;
      } else {
        int b, tok;
        dst = (c.b < 0 ? p.ws_pre_o : p.out) + (long long)c.out_row(p, row - first, b, tok) * D;
      }
      // (a lane's row is its own: 16-byte pieces of 128 rows took 4900 cycles)
      const float* v = reinterpret_cast<const float*>(acc);
      if (reinterpret_cast<uintptr_t>(dst) % 32 == 0) {
#pragma unroll
        for (int i = 0; i < C; i += 8) store_f32x8(dst + col + i, v + i);
      } else {
#pragma unroll
        for (int i = 0; i < C; i += 4)
          *reinterpret_cast<float4*>(dst + col + i) =
              make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
  }
}

// ------------------------------------------------------------------ MMA warps
// One warp issues the scores' products and another the values', so that
// one's waits do not hold up the other's.  All lanes walk the tiles, with values the compiler can
// see to be the same in all of them, and one issues: the operands then live in uniform
// registers (moved there one by one by a single lane, an MMA took 100 cycles
// to issue, three times what a 128 x 64 x 16 one takes to run).  The low terms go first: their
// steps truncate at their own size.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// A place that goes round `n` of them, and how often it went round, modulo 2.
struct Round {
  int at = 0;
  uint32_t odd = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) {
      at = 0;
      odd ^= 1;
    }
  }
};
// Both waits; asked for together, so that where both are over they cost one's latency.
template <int D>
__device__ __forceinline__ bool warp_wait2(const PrefixParams& p, PrefixSmem<D>& s, uint64_t* a,
                                           uint32_t pa, uint64_t* b, uint32_t pb) {
  const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
  if (__all_sync(0xffffffffu, x && y)) return true;
  return warp_wait<D>(p, s, a, pa) && warp_wait<D>(p, s, b, pb);
}

template <int D>
__device__ void qk_loop(const PrefixParams& p, PrefixSmem<D>& s) {
  using G = PGeo<D>;
  constexpr int KT = G::KT;
  constexpr uint32_t idesc = f16_idesc(KT, false);
  const uint32_t tm = uniform(s.tmem);
  const uint64_t q = smem_desc(smem_u32(s.q), 16, 1024);  // all 128 rows, whoever's they are
  const uint64_t k0 = smem_desc(smem_u32(s.ring), 16, 1024);
  int x = 0;
  uint32_t odd = 0;  // by barrier of q_full: parity of the uses so far
  Round buf, ring;
  for (Cursor<D> c(p, s); c.step();) {
    const int n = uniform(c.n), set = uniform(c.set());
    const int part = G::QT ? set : uniform(c.k) & 1;
    if (!warp_wait<D>(p, s, &s.q_full[part], (G::QT ? odd >> part : c.k >> 1) & 1)) return;
    odd ^= 1u << part;
    for (int j = 0; j < n; ++j, ++x) {
      int slot = ring.at;
      uint32_t use = ring.odd;
      if constexpr (!G::QT) {
        const Place<D> at = Place<D>::k(x);
        slot = at.slot;
        use = at.use & 1;
      }
      // the buffer's last tile: its products are done and its factor is read
      if constexpr (G::QT) {
        // (the first time round the other parity, which has always passed)
        if (!warp_wait2<D>(p, s, &s.b_free[buf.at], buf.odd ^ 1, &s.full[slot], use)) return;
      } else {
        // before the wait for K: in a shared ring of three the slot held that tile's V, and only
        // then has its phase passed that the next one's parity is told from
        if (!warp_wait<D>(p, s, &s.b_free[buf.at], buf.odd ^ 1)) return;
        if (!warp_wait<D>(p, s, &s.full[slot], use)) return;
      }
      tc5_fence_after();
      const uint64_t k = k0 + slot * (G::TILE / 16);
      const uint32_t d = tm + G::S0 + buf.at * KT;
      if (elect_one()) {
#pragma unroll G::QT ? 2 * G::SL : 1  // D = 256: its descriptors would spill
        for (int i = 0; i < 2 * G::SL; ++i) {
          const int term = i < G::SL ? 1 : 0, slice = i < G::SL ? i : i - G::SL;
#pragma unroll
          for (int u = 0; u < 4; ++u) {  // 16 values: 32 bytes, 8 columns
            const uint64_t kd = k + slice * (KT * 128 / 16) + u * 2;
            if constexpr (G::QT)
              mma_ts(d, tm + G::Q0 + term * (D / 2) + slice * 32 + u * 8, kd, idesc, i + u > 0);
            else
              mma_ss(d, q + (term * G::QTERM + slice * (kPrefixRows * 128)) / 16 + u * 2, kd, idesc,
                     i + u > 0);
          }
        }
        mma_commit(&s.s_full[set * G::NS + buf.at]);
        mma_commit(&s.empty[slot]);
        if (j == n - 1) mma_commit(&s.q_free[part]);
      }
      __syncwarp();
      buf.next(G::NS);
      ring.next(G::RK);
    }
  }
}

template <int D>
__device__ void pv_loop(const PrefixParams& p, PrefixSmem<D>& s) {
  using G = PGeo<D>;
  constexpr int KT = G::KT;
  constexpr uint32_t idesc = f16_idesc(D, true);
  const uint32_t tm = uniform(s.tmem);
  const uint64_t v0 = smem_desc(smem_u32(s.ring), KT * 128, 1024);
  int x = 0;
  uint32_t groups = 0;
  Phases<D> phases;  // of p_full
  Round buf, ring;
  for (Cursor<D> c(p, s); c.step();) {
    const int n = uniform(c.n), set = uniform(c.set() * G::NS);
    for (int j = 0; j < n; ++j, ++x) {
      const int at_p = set + buf.at;
      const uint32_t parity = G::QT ? phases.next(at_p, x) : buf.odd;
      int slot = G::RK + ring.at;
      uint32_t use = ring.odd;
      if constexpr (G::QT) {
        if (!warp_wait2<D>(p, s, &s.full[slot], use, &s.p_full[at_p], parity)) return;
      } else {
        // V last: in a shared ring of three the slot held this tile's K
        const Place<D> at = Place<D>::v(x);
        slot = at.slot;
        use = at.use & 1;
        if (!warp_wait<D>(p, s, &s.p_full[at_p], parity)) return;
        if (!warp_wait<D>(p, s, &s.full[slot], use)) return;
      }
      const bool start =
          j % kGroup == 0 || uniform(*reinterpret_cast<const int*>(s.grew[buf.at])) != 0;
      if (start && groups > 0 && !warp_wait<D>(p, s, &s.o_free, (groups - 1) & 1)) return;
      groups += start;
      tc5_fence_after();
      const uint64_t v = v0 + slot * (G::TILE / 16);
      const uint32_t a = tm + G::S0 + buf.at * KT;
      if (elect_one()) {
#pragma unroll
        for (int term = 1; term >= 0; --term)
#pragma unroll
          for (int k = 0; k < KT; k += 16)
            mma_ts(tm, a + k / 32 * 32 + term * 16 + k % 32 / 2, v + k * 8, idesc,
                   term == 0 || k > 0 || !start);
        mma_commit(&s.pv_done[at_p]);
        mma_commit(&s.b_free[buf.at]);
        mma_commit(&s.empty[slot]);
      }
      __syncwarp();
      buf.next(G::NS);
      ring.next(G::QT ? G::RV : 1);
    }
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
      mbar_init(&s.b_free[i], 1 + 4 * G::SUMG);
    }
    for (int i = 0; i < G::SETS * G::NS; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], i < (G::SETS - 1) * G::NS ? 1 : 4);
      mbar_init(&s.pv_done[i], 1);
    }
    mbar_init(&s.o_free, 4 * G::SUMG);
    for (int i = 0; i < (G::QT ? G::SETS : 2); ++i) {
      // Q in tensor memory: two or eight warps load it, the products use it; else one group's
      // four warps and warp 3 load it, the products use it and the group reads its row_scale
      mbar_init(&s.q_full[i], !G::QT ? 5 : i < 4 ? 2 : 8);
      mbar_init(&s.q_free[i], G::QT ? 1 : 5);
    }
    mbar_init(&s.drain[0], 1);
    mbar_init(&s.drain[1], 1);
    for (int i = 0; i < (G::QT ? kParts : 0); ++i) mbar_init(&s.part_ready[i], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s.m_ready[i], 1);
      mbar_init(&s.l_ready[0][i], 1);
      mbar_init(&s.l_ready[1][i], 1);
      mbar_init(&s.q_half[i], 2);
    }
    fence_mbarrier_init();
    s.lo = 0x7fffffff;
    s.hi = 0;
    s.plan.width = 1;
    s.best = ~0ull;
    s.abort = 0;
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
  }
  if (warp == 1) tmem_alloc(&s.tmem, 512);
  let_next_grid_start();
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  wait_for_grid_before();
  const int flags = make_plan<D>(p, s);
  if (blockIdx.x == 0 && flags && p.dev_status) atomicOr(p.dev_status, flags);
  share_out<D>(p, s);
  __syncthreads();
  if (blockIdx.x == 0) {
    if (tid == 0) *reinterpret_cast<PrefixPlan*>(p.ws_plan) = s.plan;
    for (int i = tid; i <= p.B; i += G::THREADS) p.ws_plan[kPlanInts + i] = s.cum[i];
  }
  if (warp < 4) {
    setmaxnreg_dec<G::REG_LOAD>();
    if (warp == 0 || (warp == 3 && G::QT)) {
      Loader<D> ld(p, s);
      if constexpr (!G::QT)
        ld.run_both();
      else if (warp == 0)
        ld.template run_one<G::RK, Lister<D, true>>(false, 0);
      else
        ld.template run_one<G::RV, Cursor<D>>(true, G::RK);
      const int bad = __reduce_or_sync(0xffffffffu, ld.flags);
      if (bad && lane == 0 && p.dev_status) atomicOr(p.dev_status, bad);
      if (*(volatile int*)&s.abort) ld.drain();
    } else if (warp < 3) {
      if (warp == 1)
        qk_loop<D>(p, s);
      else
        pv_loop<D>(p, s);
      if (lane == 0 && *(volatile int*)&s.abort) {
        // the products in flight end before their memory is given back
        mma_commit(&s.drain[warp - 1]);
        mbar_wait(&s.drain[warp - 1], 0, nullptr, p.wait_ns);
      }
    } else {
      if constexpr (!G::QT) q_loop<D>(p, s);
    }
  } else if (warp < 4 + 4 * G::SOFTG) {
    if constexpr (G::REG_SOFT > G::REG_LAUNCH)
      setmaxnreg_inc<G::REG_SOFT>();
    else
      setmaxnreg_dec<G::REG_SOFT>();
    if constexpr (G::QT)
      softmax_loop_two<D, CAP>(p, s);
    else
      softmax_loop_one<D, CAP>(p, s);
  } else {
    setmaxnreg_inc<G::REG_SUM>();
    sum_loop<D>(p, s);
  }
  __syncwarp();
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  if (tid == 0 && s.abort && p.dev_status) atomicOr(p.dev_status, DEV_TIMEOUT);
  if (warp == 1) tmem_free(s.tmem, 512);
}

// ------------------------------------------------------------------ joining the states
constexpr int kMergeWarps = 8;

template <int V>
__device__ __forceinline__ void load_row(const float* p, float* x) {
  if constexpr (V == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    x[0] = f.x, x[1] = f.y;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
    }
  }
}

// One warp a row: a lane finds and weighs a state, the warp adds their rows up.  Bound by a chain
// of loads (plan, (m, l), o): 5 us behind the first kernel's end for 1024 rows, 10 for 8192.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    prefix_merge_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const long long at = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  let_next_grid_start();
  wait_for_grid_before();
  if (at >= (long long)p.B * p.T * p.Hq) return;
  const int row = (int)at;
  const int bt = row / p.Hq, hq = row - bt * p.Hq, h = hq / p.G;
  const int b = bt / p.T, tok = bt - b * p.T;
  const int r1 = tok * p.G + hq - h * p.G;
  const int rb = b * p.R1 + r1;
  const PrefixPlan plan = *reinterpret_cast<const PrefixPlan*>(p.ws_plan);
  const int* cum = p.ws_plan + kPlanInts;
  const Split pre(plan.pre_share, plan.pre_rem), front(plan.first_share, plan.first_rem),
              rest(plan.rest_share, plan.rest_rem);
  // the groups of CTAs that hold the row's prefix unit
  const int n0 = plan.pn, rt = rb / kPrefixRows, block = (uint32_t)rt / (uint32_t)plan.width;
  const int g0 = (h * plan.blocks + block) * n0;
  const int c0 = n0 ? pre.cta(g0 + kPrefixExtra<D>) : 0;
  const int s0 = n0 ? pre.cta(g0 + n0 - 1) - c0 + 1 : 0;  // its states
  // the CTAs that hold its own unit
  auto own_at = [&](int g) {  // place among them of the one that holds entry g
    return g < plan.before ? front.cta(g) : plan.others + rest.cta(g - plan.before);
  };
  const int n1 = cum[b + 1] - cum[b];
  const int g1 = cum[b] * (p.Hkv * p.own_tiles) + (h * p.own_tiles + r1 / kPrefixRows) * n1;
  const int c1 = n1 ? own_at(g1 + kOwnExtra) : 0;
  const int s1 = n1 ? own_at(g1 + n1 - 1) - c1 + 1 : 0;
  float M = -kInf, L = 0.f, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int j0 = 0; j0 < s0 + s1; j0 += 32) {
    // a lane finds and weighs one state
    const int j = j0 + lane;
    const float2* ml = nullptr;
    const float* src = nullptr;
    if (j < s0 + s1) {
      const bool own = j >= s0;
      const int states = own ? s1 : s0, jj = own ? j - s0 : j, first = own ? c1 : c0;
      if (states == 1) {
        ml = (own ? p.ws_own_ml : p.ws_pre_ml) + row;
        src = (own ? p.out : p.ws_pre_o) + (long long)row * D;
      } else {
        // in the first CTA's second place if its run began before the unit
        int c = first + jj;
        long long at;
        if (own) {
          const int start =
              c < plan.others ? front.start(c) : plan.before + rest.start(c - plan.others);
          c = c < plan.others ? plan.members + c : c - plan.others;
          at = (long long)p.grid * (2 * kPrefixRows) +
               (2 * c + (jj == 0 && start < g1 ? 1 : 0)) * p.own_rows + r1 % kPrefixRows;
        } else {
          at = (long long)(2 * (c * plan.width + rt - block * plan.width) +
                           (jj == 0 && pre.start(c) < g0 ? 1 : 0)) *
                   kPrefixRows +
               rb % kPrefixRows;
        }
        ml = p.ws_cut_ml + at;
        src = p.ws_cut_o + at * D;
      }
    }
    const float2 v = ml ? *ml : make_float2(-kInf, 0.f);
    const bool some = v.y != 0.f;  // has a key
    float top = some ? v.x : -kInf;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float mn = fmaxf(M, top);
    if (mn == -kInf && !__any_sync(0xffffffffu, some)) continue;
    const float f = ex2_ftz(M - mn), w = some ? ex2_ftz(v.x - mn) : 0.f;
    float l = w * v.y;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    L = fmaf(L, f, l);
    M = mn;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] *= f;
    // their rows, several in flight (places behind the last name the last one)
    const int n = min(32, s0 + s1 - j0);
    const uint32_t have = __ballot_sync(0xffffffffu, some);
    auto add = [&](int u0, auto batch) {
      constexpr int N = decltype(batch)::value;
      float x[N][V];
#pragma unroll
      for (int u = 0; u < N; ++u)
        load_row<V>(reinterpret_cast<const float*>(__shfl_sync(
                        0xffffffffu, reinterpret_cast<unsigned long long>(src),
                        min(u0 + u, n - 1))) + lane * V, x[u]);
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, (u0 + u) & 31);
        if (u0 + u < n && (have >> (u0 + u) & 1)) {
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = fmaf(wu, x[u][i], o[i]);
        }
      }
    };
    int u0 = 0;
#pragma unroll 1
    for (; n - u0 > 4; u0 += 8) add(u0, std::integral_constant<int, 8>());
    if (u0 < n) add(u0, std::integral_constant<int, 4>());
  }
  // A masked key's weight of zero does not silence a value that is not finite, and two terms make NaN
  // of an infinite product that one would leave infinite: a row that came out non-finite is done
  // again, key by key.
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) bad |= !isfinite(o[i]);
  if (__any_sync(0xffffffffu, bad)) {
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
  err = launch_early(prefix_attn_kernel<D, CAP>, p.grid, PGeo<D>::THREADS, smem, stream, p);
  if (err != cudaSuccess) return err;
  return launch_early(prefix_merge_kernel<D>, (unsigned)blocks, kMergeWarps * 32, 0, stream, p);
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
