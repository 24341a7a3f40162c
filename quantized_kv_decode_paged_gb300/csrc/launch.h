// launch.h — host-side entry points into the kernel translation units.
#pragma once

#include <cuda_runtime.h>

#include "../../include/decode_attn.h"
#include "kernel_params.h"

namespace da {

// Validation of the geometry an append uses (append.cu).
int check_append_params(const da_params* p);

// Validation of a page format in 4 bits (q4.cu).
int check_q4(const da_params* p, int group);

// Validation of da_params as the paged decode entry points do it; the score scale in base-2
// units (api.cu).
int check_paged(const da_params* p);
float base2_scale(const da_params* p);

// SM count of the current device (api.cu); a status.
int device_sms(int* sms_out);

// kv heads per work unit for a cache of `kind` with head dimension D and
// Hkv kv heads: enough that one token row of the block is >= 512
// contiguous bytes, and a divisor of Hkv.
inline int decode_kvb(int kind, int D, int Hkv) {
  int pref = cold_int8(kind) ? (D == 128 ? 4 : 2) : (D == 64 ? 4 : D == 128 ? 2 : 1);
  while (pref > 1 && Hkv % pref != 0) pref /= 2;
  return pref;
}

// Geometry numbers of the instantiation (kind, D, KVB) for the host.
struct GeoInfo {
  int W, TOK, TOKH, REGION, THREADS;
};
GeoInfo decode_geo(int kind, int D, int KVB);

// Launches the decode kernel of (kind, D, KVB); `packed` selects the variant
// that packs the f16 and remainder parts of Q and P into one MMA operand
// (valid when p.NH <= 4).  Returns cudaErrorInvalidValue for a combination
// that has no instantiation.
cudaError_t launch_decode(int kind, int D, int KVB, bool packed, const KParams& p, dim3 grid,
                          int smem_bytes, cudaStream_t stream);

// Bytes at the start of a stream-K workspace that hold the ticket counters
// on the current device (they must be zero when a call starts); 0 when the
// device cannot be queried.
size_t workspace_ticket_bytes();

// out/lse from max_splits partial states per (b, h).
cudaError_t launch_split_merge(int rows, int max_splits, int D, const float* o_part,
                               const float* lse_part, float* out, float* lse,
                               cudaStream_t stream);

// Launches a kernel that may be set up while the kernel before it in the stream still runs, and
// that waits for that one's end itself (wait_for_grid_before) before it touches memory.
template <typename P>
inline cudaError_t launch_early(void (*kernel)(const P), unsigned grid, unsigned threads,
                                size_t smem, cudaStream_t stream, const P& p) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Shared-prefix decode (prefix_attn.cu).  Rows are (sequence, query token,
// query head of the kv head); keys below prefix_pages * bs are read through
// prefix_table, the others through block_table.
constexpr int kPrefixRows = 128;      // rows of a tile (the MMA's M)
// sequences of a launch: their lengths sit in shared memory beside the tiles
__host__ __device__ constexpr int prefix_max_batch(int D) { return D >= 256 ? 144 : 256; }
// keys of a tile
__host__ __device__ constexpr int prefix_tile_keys(int D) { return D == 64 ? 128 : 64; }

struct alignas(128) PrefixParams {
  CUtensorMap tm_k;  // boxes of box_rows keys, one kv head, box_slices 128-byte slices
  CUtensorMap tm_v;
  int box_rows, box_slices;
  int B, T, Hq, Hkv, D, G;
  int R1;             // rows of a sequence and kv head: T * G
  int row_tiles;      // tiles of the batch's rows of a kv head
  int own_tiles;      // tiles of one sequence's rows of a kv head
  int own_rows;       // most rows of such a tile
  int bs, log2_bs, max_blocks, num_blocks;
  int prefix_pages;
  int window, causal;
  float qscale;       // scale * log2(e): scores are kept in base-2 units
  float softcap2;     // softcap * log2(e) (0 = off)
  float softcap_inv;  // 1 / softcap2
  int grid;
  unsigned long long wait_ns;  // time limit of every wait (abort mode after it)
  int test_skip_arm;           // test hook: the first copy is left out
  const float* q;
  const uint16_t* k_pool;
  const uint16_t* v_pool;
  const int* prefix_table;
  const int* block_table;
  const int* seq_lens;
  const int* q_pos;
  float* out;
  float* lse;
  int* dev_status;
  // workspace (PrefixWs).  A state is o (not divided by l), and (m, l): the
  // reference the weights were taken against, base 2, and their sum.
  int* ws_plan;       // PrefixPlan, then [B + 1] entries of the own list before b's
  float2* ws_cut_ml;  // [grid][2][128] of a prefix unit's part, [grid][2][own_rows] of an own one's
  float2* ws_pre_ml;  // [B * T * Hq] of the prefix, units that no CTA boundary cuts
  float2* ws_own_ml;  // [B * T * Hq] of own keys; their o goes to out
  float* ws_cut_o;    // as ws_cut_ml, [D]
  float* ws_pre_o;    // [B * T * Hq][D]
};

// How the work is shared out, as prefix_attn_kernel decides it and prefix_merge_kernel reads it.
struct PrefixPlan {
  int pn;                     // entries of a prefix unit
  int width, blocks;          // tiles of rows that CTAs work on side by side; blocks of so many
  int pre_share, pre_rem;     // of the groups of `width` CTAs: the prefix's Split
  int members, others;        // CTAs of the groups; those behind them, which take the own
  int before;                 // list's first entries
  int first_share, first_rem;  // the Split of these
  int rest_share, rest_rem;   // and of the others, among the members
};

struct PrefixWs {
  size_t plan, cut_ml, pre_ml, own_ml, cut_o, pre_o, total;
};
inline PrefixWs prefix_ws(int grid, int D, long long rows, int own_rows) {
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  PrefixWs w;
  w.plan = 0;
  const size_t cut_rows = (size_t)grid * 2 * (kPrefixRows + own_rows);
  w.cut_ml = al(sizeof(PrefixPlan) + (prefix_max_batch(D) + 1) * 4);
  w.pre_ml = w.cut_ml + al(cut_rows * 8);
  w.own_ml = w.pre_ml + al((size_t)rows * 8);
  w.cut_o = w.own_ml + al((size_t)rows * 8);
  w.pre_o = w.cut_o + al(cut_rows * D * 4);
  w.total = w.pre_o + al((size_t)rows * D * 4);
  return w;
}
cudaError_t launch_prefix(const PrefixParams& p, cudaStream_t stream);

}  // namespace da
