// plan.cu — pages for requests whose lengths change, and the places of their new tokens.
//
// With po = ceil(old / bs) and pn = ceil(new / bs) pages before and after, a request that grows takes
// pn - po pages, one that shrinks gives po - pn back and one that gains tokens has places for
// them.  Free pages are a stack: those given back go on top in the order of requests and of
// their pages, then the top T are taken, the lowest of them first.  So whoever takes page k of the
// call takes entry left + k of the stack, left being what remains, and undoing a call (old and
// new exchanged) puts every page back where it was.
//
// The three running sums over the requests are all that the rest depends on: every CTA works them
// out for itself in shared memory, and its threads then go through pages and tokens by
// binary searches in them.  Nothing is changed before all that the call reads is known
// to be sound, and entries given back are cleared when nobody reads them any more; the two
// barriers that this takes are a cluster's, so the whole call is one launch of one cluster.
// Latency bounds it: the chain of loads (lengths, table, stack) and the sums.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/decode_attn.h"
#include "launch.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 1024;
// CTAs of a large call (8 where no cluster of 16 fits): a call that takes 101,000 pages back and places 20,000 tokens
// takes 36 us with 8 and 23 with 16.
constexpr int kCluster = 16;
constexpr int kMaxBatch = 16384;   // three sums of each in shared memory
constexpr int kKeptBatch = 10240;  // both lengths too
constexpr size_t kOwnShared = 1024;  // at most, of shared memory that the kernel declares
// A warp takes up to 32 * kRun entries side by side: most are the request's that the one before was, and need no
// search, and their loads are under way together (the same call, with 8 CTAs: 42 us with one entry at a time).
constexpr int kRun = 8;

struct PlanArgs {
  int B, log2_bs, max_blocks, num_blocks, max_tokens, free_capacity, ctas;
  const int32_t* old_lens;
  const int32_t* new_lens;
  int32_t* table;
  int32_t* free_list;
  int32_t* free_count;
  int32_t* positions;
  int32_t* token_seq;
  long long* slots;
  int32_t* cu;
  int32_t* dev_status;
};

struct Sums {
  long long tokens, taken, given;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.tokens + b.tokens, a.taken + b.taken, a.given + b.given};
}
__device__ __forceinline__ Sums shfl_up(const Sums& a, int by) {
  return {__shfl_up_sync(0xffffffffu, a.tokens, by), __shfl_up_sync(0xffffffffu, a.taken, by),
          __shfl_up_sync(0xffffffffu, a.given, by)};
}

// The request that entry i of a running sum belongs to: the last b with sum[b] <= i (entries of
// requests without any are passed over).
__device__ __forceinline__ int find(const int* sum, int B, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (sum[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same where b is the request of an earlier entry.
__device__ __forceinline__ int find_from(const int* sum, int B, int i, int b) {
  return sum[b + 1] > i ? b : find(sum, B, i);
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
  extern __shared__ int smem[];
  __shared__ Sums warp_sums[kThreads / 32];
  __shared__ int flags, flags_found;  // of lengths and counts; of what table and stack hold
  static_assert(sizeof(warp_sums) + 2 * sizeof(int) + 16 <= kOwnShared, "shared memory");
  cg::cluster_group cluster = cg::this_cluster();
  int* cu = smem;                // [B + 1] tokens before request b
  int* taken = cu + a.B + 1;     // pages taken before it
  int* given = taken + a.B + 1;  // pages given back before it
  const bool keep = a.B <= kKeptBatch;
  int* kept = given + a.B + 1;  // [2][B] lengths before and after
  const int* old_lens = keep ? kept : a.old_lens;
  const int* new_lens = keep ? kept + a.B : a.new_lens;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x;
  const int bs = 1 << a.log2_bs;
  const long long cap = (long long)a.max_blocks << a.log2_bs;
  if (tid == 0) flags = flags_found = 0;
  __syncthreads();
  cluster.barrier_arrive();  // waited for before another CTA's flag is written

  // the sums: a thread has `per` requests side by side
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  if (keep) {
    for (int b = tid; b < a.B; b += kThreads) {
      kept[b] = a.old_lens[b];
      kept[a.B + b] = a.new_lens[b];
    }
    __syncthreads();
  }
  int bad = 0;
  auto of = [&](int b) {
    const long long o = old_lens[b], n = new_lens[b];
    if (o < 0 || n < 0 || o > cap || n > cap) {
      bad |= DA_DEV_BAD_SEQ_LEN;
      return Sums{0, 0, 0};
    }
    const long long po = (o + bs - 1) >> a.log2_bs, pn = (n + bs - 1) >> a.log2_bs;
    return Sums{n > o ? n - o : 0, pn > po ? pn - po : 0, po > pn ? po - pn : 0};
  };
  Sums mine = {0, 0, 0};
  for (int b = b0; b < b1; ++b) mine = mine + of(b);
  Sums upto = mine;
#pragma unroll
  for (int by = 1; by < 32; by <<= 1) {
    const Sums below = shfl_up(upto, by);
    if (lane >= by) upto = upto + below;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    Sums w = warp_sums[lane];
#pragma unroll
    for (int by = 1; by < 32; by <<= 1) {
      const Sums below = shfl_up(w, by);
      if (lane >= by) w = w + below;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const Sums all = warp_sums[kThreads / 32 - 1];
  Sums run = warp ? warp_sums[warp - 1] : Sums{0, 0, 0};
  run = {run.tokens + upto.tokens - mine.tokens, run.taken + upto.taken - mine.taken,
         run.given + upto.given - mine.given};
  for (int b = b0; b < b1; ++b) {
    cu[b] = (int)run.tokens;
    taken[b] = (int)run.taken;
    given[b] = (int)run.given;
    run = run + of(b);
  }
  if (tid == 0) {
    cu[a.B] = (int)all.tokens;
    taken[a.B] = (int)all.taken;
    given[a.B] = (int)all.given;
  }
  const long long count = *a.free_count;
  const int most_free = min(a.free_capacity, a.num_blocks);
  if (count < 0 || count > most_free) bad |= DA_DEV_BAD_FREE_LIST;
  if (all.tokens > a.max_tokens) bad |= DA_DEV_TOKEN_OVERFLOW;
  if (all.given > a.num_blocks) bad |= DA_DEV_BAD_BLOCK;  // a page is held twice
  const long long left64 = count + all.given - all.taken;
  if (left64 < 0) bad |= DA_DEV_NO_BLOCKS;
  if (left64 > most_free) bad |= DA_DEV_BAD_FREE_LIST;
  if (bad) atomicOr(&flags, bad);
  __syncthreads();
  const bool sound = flags == 0;  // the same in every CTA

  const int step = a.ctas * kThreads, first = rank * kThreads + tid;
  const int T = (int)all.taken, R = (int)all.given, N = (int)all.tokens;
  const int F = (int)count, left = (int)left64;
  auto pages = [&](int len) { return (len + bs - 1) >> a.log2_bs; };
  // table entry of page i of those given back; b: the request of an earlier one, and this one's
  auto given_at = [&](int i, int& b) {
    b = find_from(given, a.B, i, b);
    return (long long)b * a.max_blocks + pages(new_lens[b]) + (i - given[b]);
  };
  // the page that entry k of those taken gets
  auto taken_page = [&](int k, int& b) {
    const int i = left + k;
    return i < F ? a.free_list[i] : a.table[given_at(i - F, b)];
  };
  // each entry of `count` once: use(i, load(i)), the loads of a run before the first use
  auto each = [&](int count, auto load, auto use) {
    const int run = min(kRun, (count + step - 1) / step);
    for (int i0 = (rank * (kThreads / 32) + warp) * (32 * run) + lane; i0 - lane < count;
         i0 += step * run) {
      decltype(load(0)) x[kRun];
#pragma unroll
      for (int u = 0; u < kRun; ++u)
        if (u < run && i0 + 32 * u < count) x[u] = load(i0 + 32 * u);
#pragma unroll
      for (int u = 0; u < kRun; ++u)
        if (u < run && i0 + 32 * u < count) use(i0 + 32 * u, x[u]);
    }
  };
  auto is_page = [&](int id) { return id >= 0 && id < a.num_blocks; };

  cluster.barrier_wait();
  if (sound) {
    // all that is read from table and stack: pages given back, pages taken, last pages that grow
    bad = 0;
    int g = 0;
    each(R, [&](int i) { return a.table[given_at(i, g)]; },
         [&](int, int id) {
           if (!is_page(id)) bad |= DA_DEV_BAD_BLOCK;
         });
    for (int i = left + first; i < F; i += step)
      if (!is_page(a.free_list[i])) bad |= DA_DEV_BAD_FREE_LIST;
    for (int b = first; b < a.B; b += step) {
      const int o = old_lens[b];
      if (new_lens[b] > o && (o & (bs - 1)) &&
          !is_page(a.table[(long long)b * a.max_blocks + (o >> a.log2_bs)]))
        bad |= DA_DEV_BAD_BLOCK;
    }
    if (bad)
      for (int c = 0; c < a.ctas; ++c) atomicOr(cluster.map_shared_rank(&flags_found, c), bad);
  }
  cluster.sync();
  const int found = flags | flags_found;
  if (found) {
    // nothing is changed; the outputs are all padding
    for (int n = first; n < a.max_tokens; n += step) {
      a.positions[n] = 0;
      a.token_seq[n] = -1;
      a.slots[n] = -1;
    }
    for (int b = first; b <= a.B; b += step) a.cu[b] = 0;
    if (first == 0 && a.dev_status) atomicOr(a.dev_status, found);
  } else {
    int g = 0, t = 0;
    each(T, [&](int k) { return taken_page(k, g); },
         [&](int k, int id) {
           t = find_from(taken, a.B, k, t);
           a.table[(long long)t * a.max_blocks + pages(old_lens[t]) + (k - taken[t])] = id;
         });
    struct Token {
      int seq, pos, id;
    };
    int b = 0;
    g = 0;
    each(a.max_tokens,
         [&](int n) {
           Token x = {-1, 0, -1};
           if (n < N) {
             x.seq = b = find_from(cu, a.B, n, b);
             const int o = old_lens[b], held = pages(o);
             x.pos = o + (n - cu[b]);
             const int page = x.pos >> a.log2_bs;
             x.id = page < held ? a.table[(long long)b * a.max_blocks + page]
                                : taken_page(taken[b] + page - held, g);
           }
           return x;
         },
         [&](int n, const Token& x) {
           a.positions[n] = x.pos;
           a.token_seq[n] = x.seq;
           a.slots[n] = x.seq < 0 ? -1 : ((long long)x.id << a.log2_bs) + (x.pos & (bs - 1));
         });
    for (int i = first; i <= a.B; i += step) a.cu[i] = cu[i];
  }
  // every CTA is past its reads of entries that change now (and of the others' flags)
  cluster.sync();
  if (found) return;
  struct Entry {
    long long at;
    int id;
  };
  int g = 0;
  each(R,
       [&](int i) {
         const long long at = given_at(i, g);
         return Entry{at, F + i < left ? a.table[at] : -1};
       },
       [&](int i, const Entry& x) {
         if (F + i < left) a.free_list[F + i] = x.id;
         a.table[x.at] = -1;
       });
  if (first == 0) *a.free_count = left;
}

// CTAs of a large call on the current device: as many as its processors side by side can hold.
cudaError_t large_cluster(int* ctas) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::atomic<int>& n = known[dev % 64];
  if ((*ctas = n.load(std::memory_order_relaxed))) return cudaSuccess;
  err = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)kCluster, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  err = cudaOccupancyMaxActiveClusters(&clusters, plan_kernel, &cfg);
  if (err != cudaSuccess) return err;
  *ctas = clusters > 0 ? kCluster : 8;
  n.store(*ctas, std::memory_order_relaxed);
  return cudaSuccess;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" int decode_attn_plan_blocks(int32_t batch, int32_t block_size,
                                       int32_t max_blocks_per_seq, int32_t num_blocks,
                                       int32_t max_tokens, int32_t free_capacity,
                                       const int32_t* old_lens, const int32_t* new_lens,
                                       int32_t* block_table, int32_t* free_list,
                                       int32_t* free_count, int32_t* positions,
                                       int32_t* token_seq, int64_t* slots, int32_t* cu_tokens,
                                       int32_t* dev_status, void* stream) {
  if (batch < 0 || block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
      max_tokens < 0 || free_capacity < 0)
    return DA_ERR_INVALID;
  if ((block_size & (block_size - 1)) != 0 || block_size < 8 || block_size > 256)
    return DA_ERR_UNSUPPORTED;
  if ((long long)num_blocks * block_size > 0x7fffffffLL ||
      (long long)max_blocks_per_seq * block_size > 0x7fffffffLL || batch > kMaxBatch ||
      max_tokens > 0x7fffffff - (1 << 21) || free_capacity > 0x7fffffff - (1 << 21))
    return DA_ERR_UNSUPPORTED;
  if (!old_lens || !new_lens || !block_table || !free_count || !cu_tokens ||
      (free_capacity > 0 && !free_list) ||
      (max_tokens > 0 && (!positions || !token_seq || !slots)))
    return DA_ERR_INVALID;
  for (const void* p : {(const void*)old_lens, (const void*)new_lens, (const void*)block_table,
                        (const void*)free_list, (const void*)free_count, (const void*)positions,
                        (const void*)token_seq, (const void*)cu_tokens, (const void*)dev_status})
    if (!aligned(p, 4)) return DA_ERR_INVALID;
  if (!aligned(slots, 8)) return DA_ERR_INVALID;
  if (batch == 0 && max_tokens == 0) return DA_OK;
  PlanArgs a = {};
  a.B = batch;
  while ((1 << a.log2_bs) < block_size) ++a.log2_bs;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.max_tokens = max_tokens;
  a.free_capacity = free_capacity;
  a.old_lens = old_lens;
  a.new_lens = new_lens;
  a.table = block_table;
  a.free_list = free_list;
  a.free_count = free_count;
  a.positions = positions;
  a.token_seq = token_seq;
  a.slots = reinterpret_cast<long long*>(slots);
  a.cu = cu_tokens;
  a.dev_status = dev_status;
  const size_t smem = 3 * sizeof(int) * ((size_t)batch + 1) +
                      (batch <= kKeptBatch ? 2 * sizeof(int) * (size_t)batch : 0);
  constexpr size_t kMost = 5 * sizeof(int) * kKeptBatch + 64;
  static_assert(kMost >= 3 * sizeof(int) * (kMaxBatch + 1) && kMost + kOwnShared <= 227 * 1024,
                "shared memory");
  // what a kernel has without being allowed more, its own included
  if (smem + kOwnShared > 48 * 1024 &&
      cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) !=
          cudaSuccess)
    return DA_ERR_CUDA;
  // one CTA where its threads have at most a token or a request each
  a.ctas = 1;
  if ((batch > kThreads || max_tokens > kThreads) && large_cluster(&a.ctas) != cudaSuccess)
    return DA_ERR_CUDA;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)a.ctas, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, a) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}
