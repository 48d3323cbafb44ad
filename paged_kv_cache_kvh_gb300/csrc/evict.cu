// evict.cu -- cutting sequences of the paged cache down to the tokens that attention went to.
//
// For each (sequence of n > budget tokens, kv head): the first `first` and the newest `recent` tokens stay, and of the
// others those with the largest weights (attention added up beside the cache by the decode), equal ones in order of
// position, budget in all. What stays moves up, in order: token kept[j] becomes token j.
//
// Select: one block per (sequence, kv head), or a cluster of up to 8 where there are few. Weights become unsigned numbers
// of the same order, held in shared memory (those past kCached are read again each time); three histograms of 11, 11 and
// 10 bits, each within the bin that the one before it found, summed over the cluster, give the value of the last token
// that stays and how many of its equals do. Then every warp counts what it keeps in its own stretch of positions, a scan
// over the warps (and blocks) gives each its place, and a second sweep writes kept[] in order. Counts are integers, so
// the order of the atomics changes nothing.
// (One sequence of 40007: 20 to 24 us, bound by three rounds of histogram, cluster barrier and reads of one another's
// counts; 96 sequences: 27 us.)
// Move: 512 bytes of K and V and a weight per kept token, from wherever it is to its new place; a gather bound by HBM
// (96 sequences cut to 1500: 171 us at 6.3 TB/s; one of 40007 cut to 10000: 15 to 18 us).
// To other blocks every row is on its own. In place, the rows of one (kv head, K or V, some of the 16-byte columns) belong
// to one block, which takes them in order: rows only move towards the front, so a chunk may be written once it has been
// read, and chunks behind it are still where they were (the calls in place: one of 40007 104 us, 96 sequences 266). Measured
// and not kept: rows copied by the block that has chosen them, beside the choices of others (96 sequences 229 us instead
// of 227, one of 40007 45 instead of 40: 64 SMs copy).
#include "pkv_common.cuh"

namespace pkv {

struct EvictArgs {
  void* k_cache;
  void* v_cache;
  float* weights;
  int32_t num_blocks;
  const int32_t* block_tables;
  int32_t bt_stride;
  const int32_t* context_lens;
  int32_t num_seqs, hkv, max_ctx, budget, first, recent;
  const int32_t* new_tables;  // NULL: in place
  int32_t new_stride;
  int32_t* kept;
  int32_t* new_lens;
};

namespace {

constexpr int kCached = 48 * 1024;  // tokens whose weights a block holds at most
constexpr int kBins = 2048;
constexpr int kMaxRanks = 8;        // blocks that may share a selection (a portable cluster)
constexpr int kMoveThreads = 256;
constexpr int kHalfWarps = kMoveThreads / 16;
// Rows that a half-warp has on the way, and how many times that a block copies (96 sequences cut to 1500: 1 x 8 202 us,
// 2 x 4 199, 4 x 4 214, 8 x 2 299: more rows take registers, and with them warps).
constexpr int kAhead = 2;
constexpr int kRounds = 4;

struct EvictParams {
  EvictArgs a;
  int32_t ranks;   // blocks that share a (sequence, kv head) in the selection, a cluster
  int32_t cached;  // tokens that fit in a block's shared memory
  int32_t parts;   // in place: blocks that share a row
  unsigned int* err;
};

__device__ __forceinline__ int length_of(const EvictParams& p, int b, bool report) {
  const int n = p.a.context_lens[b];
  if (n >= 0 && n <= p.a.max_ctx && n <= static_cast<int64_t>(p.a.bt_stride) * kBlockSize) return n;
  if (report) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
  return 0;
}

// The physical block of a token, or -1 (reported).
__device__ __forceinline__ int block_of(const EvictParams& p, const int32_t* tables, int stride, int b, int token) {
  const int block = tables[static_cast<int64_t>(b) * stride + token / kBlockSize];
  if (block >= 0 && block < p.a.num_blocks) return block;
  flag_error(p.err, PKV_DEVERR_BAD_BLOCK);
  return -1;
}

__device__ __forceinline__ int64_t weight_place(const EvictParams& p, int block, int hk, int token) {
  return (static_cast<int64_t>(block) * p.a.hkv + hk) * kBlockSize + token % kBlockSize;
}

// Unsigned numbers in the order of the weights; a NaN is larger than any number, zeros are equal.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (isnan(w)) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Everything that any block of the cluster wrote to shared memory before is there for all of them behind it.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Words of the same shared array in another block of the cluster.
__device__ __forceinline__ uint32_t cluster_address(const int* mine, int rank) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(mine)), "r"(rank));
  return addr;
}
__device__ __forceinline__ int cluster_load(const int* mine, int rank) {
  int x;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(cluster_address(mine, rank)) : "memory");
  return x;
}
__device__ __forceinline__ int4 cluster_load4(const int* mine, int rank) {
  int4 x;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(cluster_address(mine, rank))
               : "memory");
  return x;
}
// Sum of what the warps before this one have in x.
__device__ __forceinline__ int before_warp(const int* x, int warp, int lane) {
  return __reduce_add_sync(0xffffffffu, lane < warp ? x[lane] : 0);
}
__device__ __forceinline__ uint4 ld_row(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) int hist[];  // one of kBins, in a cluster one to a pass; then the weights
  __shared__ int s_warp[2][kWarps];
  __shared__ int s_bin, s_left, s_total[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int hists = p.ranks > 1 ? 3 : 1;
  uint32_t* keys = reinterpret_cast<uint32_t*>(hist + hists * kBins);
  const int ranks = p.ranks, rank = static_cast<int>(blockIdx.x) % ranks;
  const int hk = static_cast<int>(blockIdx.x) / ranks, b = static_cast<int>(blockIdx.y);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = length_of(p, b, blockIdx.x == 0 && tid == 0);
  const int budget = p.a.budget;
  int32_t* kept = p.a.kept + (static_cast<int64_t>(b) * p.a.hkv + hk) * budget;
  if (blockIdx.x == 0 && tid == 0) p.a.new_lens[b] = min(n, budget);
  const int all_tid = rank * kThreads + tid, all_threads = ranks * kThreads;
  if (n <= budget) {
    for (int j = all_tid; j < budget; j += all_threads) kept[j] = j < n ? j : -1;
    return;
  }
  const int all_hi = n - p.a.recent;              // the tokens to choose from: [first, all_hi)
  for (int j = all_tid; j < p.a.first; j += all_threads) kept[j] = j;
  for (int j = all_tid; j < p.a.recent; j += all_threads) kept[budget - p.a.recent + j] = all_hi + j;
  int want = budget - p.a.first - p.a.recent;     // of them
  if (want == 0) return;
  // this block's share of them
  const int share = (all_hi - p.a.first + ranks - 1) / ranks;
  const int lo = min(p.a.first + rank * share, all_hi), hi = min(lo + share, all_hi);

  const int32_t* table = p.a.block_tables + static_cast<int64_t>(b) * p.a.bt_stride;
  auto load = [&](int t) -> uint32_t {
    const int block = table[t / kBlockSize];
    if (block < 0 || block >= p.a.num_blocks) {
      if (hk == 0) flag_error(p.err, PKV_DEVERR_BAD_BLOCK);
      return 0;
    }
    return order_of(p.a.weights[weight_place(p, block, hk, t)]);
  };
  const int in_smem = min(hi, lo + p.cached);
#pragma unroll 8
  for (int t = lo + tid; t < in_smem; t += kThreads) keys[t - lo] = load(t);
  auto key = [&](int t) -> uint32_t { return t < in_smem ? keys[t - lo] : load(t); };

  for (int i = tid; i < hists * kBins; i += kThreads) hist[i] = 0;
  __syncthreads();

  // ---- the value of the last token that stays ----
  uint32_t prefix = 0, known = 0;  // the bits found so far, and their mask
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t bins = pass == 2 ? 1024u : 2048u;
    int* mine = hist + (ranks > 1 ? pass * kBins : 0);
    for (int t0 = lo + warp * 32; t0 < hi; t0 += kThreads) {
      const int t = t0 + lane;
      const uint32_t k = t < hi ? key(t) : 0u;
      const bool in = t < hi && (k & known) == prefix;
      const uint32_t bin = (k >> shift) & (bins - 1);
      // lanes that share the first one's bin (zeros, often) are added by that one
      const uint32_t all = __ballot_sync(0xffffffffu, in);
      if (all) {
        const int leader = __ffs(all) - 1;
        const uint32_t first_bin = __shfl_sync(0xffffffffu, bin, leader);
        const uint32_t same = __ballot_sync(0xffffffffu, in && bin == first_bin);
        if (lane == leader)
          atomicAdd(mine + bin, __popc(same));
        else if (in && !((same >> lane) & 1u))
          atomicAdd(mine + bin, 1);
      }
    }
    if (ranks > 1)
      cluster_sync();
    else
      __syncthreads();
    // bins from the top down, of all blocks: thread i has kBins / kThreads of them
    constexpr int kPer = kBins / kThreads < 4 ? 4 : kBins / kThreads;
    int count[kPer], total = 0;
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {  // bins of four, the last first
      int4 c = make_int4(0, 0, 0, 0);
      const int* four = mine + kBins - 4 - (tid * kPer + i);
      if (tid * kPer < kBins) {
        if (ranks == 1) {
          c = *reinterpret_cast<const int4*>(four);
        } else {
          int4 there[kMaxRanks];  // all on the way together
#pragma unroll
          for (int r = 0; r < kMaxRanks; ++r) there[r] = r < ranks ? cluster_load4(four, r) : c;
#pragma unroll
          for (int r = 0; r < kMaxRanks; ++r) {
            c.x += there[r].x;
            c.y += there[r].y;
            c.z += there[r].z;
            c.w += there[r].w;
          }
        }
      }
      count[i] = c.w;
      count[i + 1] = c.z;
      count[i + 2] = c.y;
      count[i + 3] = c.x;
      total += (c.x + c.y) + (c.z + c.w);
    }
    int scan = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, off);
      if (lane >= off) scan += y;
    }
    if (lane == 31) s_warp[0][warp] = scan;
    __syncthreads();
    const int above = scan - total + before_warp(s_warp[0], warp, lane);
    if (above < want && above + total >= want) {
      int left = want - above;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (left > 0 && left <= count[i]) {
          s_bin = kBins - 1 - (tid * kPer + i);
          s_left = left;
        }
        left -= count[i];
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_bin) << shift;
    known |= (bins - 1) << shift;
    want = s_left;
    if (ranks == 1 && pass < 2)
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
  }

  // ---- kept[]: those above the value, and the first `want` of its equals ----
  const int per_warp = ((hi - lo + kThreads - 1) / kThreads) * 32;
  const int begin = lo + warp * per_warp, end = min(hi, begin + per_warp);
  int greater = 0, equal = 0;
  for (int t0 = begin; t0 < end; t0 += 32) {
    const uint32_t k = t0 + lane < end ? key(t0 + lane) : 0u;
    const bool in = t0 + lane < end;
    greater += __popc(__ballot_sync(0xffffffffu, in && k > prefix));
    equal += __popc(__ballot_sync(0xffffffffu, in && k == prefix));
  }
  if (lane == 0) {
    s_warp[0][warp] = greater;
    s_warp[1][warp] = equal;
  }
  __syncthreads();
  int greater_before = before_warp(s_warp[0], warp, lane), equal_before = before_warp(s_warp[1], warp, lane);
  if (warp == kWarps - 1 && lane == 0) {
    s_total[0] = greater_before + s_warp[0][warp];
    s_total[1] = equal_before + s_warp[1][warp];
  }
  int greater_there = 0, equal_there = 0;  // in the blocks before this one
  if (ranks > 1) {
    cluster_sync();
    greater_there = __reduce_add_sync(0xffffffffu, lane < rank ? cluster_load(s_total, lane) : 0);
    equal_there = __reduce_add_sync(0xffffffffu, lane < rank ? cluster_load(s_total + 1, lane) : 0);
  }
  equal_before += equal_there;
  int at = p.a.first + greater_there + greater_before + min(equal_before, want);
  const uint32_t below = (1u << lane) - 1u;
  for (int t0 = begin; t0 < end; t0 += 32) {
    const bool in = t0 + lane < end;
    const uint32_t k = in ? key(t0 + lane) : 0u;
    const bool same = in && k == prefix;
    const uint32_t sames = __ballot_sync(0xffffffffu, same);
    const bool keep = in && (k > prefix || (same && equal_before + __popc(sames & below) < want));
    const uint32_t keeps = __ballot_sync(0xffffffffu, keep);
    if (keep) kept[at + __popc(keeps & below)] = t0 + lane;
    at += __popc(keeps);
    equal_before += __popc(sames);
  }
  if (ranks > 1) cluster_sync();  // no block's shared memory goes while another may read it
}

// To other blocks: an item is (kept token, kv head), heads fastest; a half-warp moves its K and V rows. The next items'
// tokens are asked for while a round's rows are on the way.
__global__ void __launch_bounds__(kMoveThreads) evict_copy_kernel(const EvictParams p) {
  const int b = static_cast<int>(blockIdx.y), hkv = p.a.hkv;
  const int lane = threadIdx.x & 15;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t items = static_cast<int64_t>(min(length_of(p, b, false), p.a.budget)) * hkv;
  int64_t item = static_cast<int64_t>(blockIdx.x) * (kHalfWarps * kAhead * kRounds) + (threadIdx.x >> 4);
  const int64_t end = min(items, static_cast<int64_t>(blockIdx.x + 1) * (kHalfWarps * kAhead * kRounds));
  uint16_t* kc = static_cast<uint16_t*>(p.a.k_cache);
  uint16_t* vc = static_cast<uint16_t*>(p.a.v_cache);
  const int32_t* kept = p.a.kept + static_cast<int64_t>(b) * hkv * p.a.budget;
  int t[kAhead], j[kAhead], hk[kAhead];
  auto ask = [&](int64_t first) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t x = first + i * kHalfWarps;
      t[i] = -1;
      if (x < end) {
        j[i] = static_cast<int>(x / hkv);
        hk[i] = static_cast<int>(x - static_cast<int64_t>(j[i]) * hkv);
        t[i] = kept[static_cast<int64_t>(hk[i]) * p.a.budget + j[i]];
      }
    }
  };
  ask(item);
  while (item < end) {
    int64_t to[kAhead], w_to[kAhead];
    uint4 k[kAhead], v[kAhead];
    float w[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      to[i] = -1;
      if (t[i] < 0) continue;
      const int from = block_of(p, p.a.block_tables, p.a.bt_stride, b, t[i]);
      const int dest = block_of(p, p.a.new_tables, p.a.new_stride, b, j[i]);
      if (from < 0 || dest < 0) continue;
      const int64_t src = ((static_cast<int64_t>(from) * kBlockSize + t[i] % kBlockSize) * hkv + hk[i]) * kHeadDim + lane * 8;
      k[i] = ld_row(kc + src);
      v[i] = ld_row(vc + src);
      w[i] = p.a.weights[weight_place(p, from, hk[i], t[i])];
      to[i] = ((static_cast<int64_t>(dest) * kBlockSize + j[i] % kBlockSize) * hkv + hk[i]) * kHeadDim + lane * 8;
      w_to[i] = weight_place(p, dest, hk[i], j[i]);
    }
    item += kHalfWarps * kAhead;
    ask(item);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (to[i] < 0) continue;
      *reinterpret_cast<uint4*>(kc + to[i]) = k[i];
      *reinterpret_cast<uint4*>(vc + to[i]) = v[i];
      if (lane == 0) p.a.weights[w_to[i]] = w[i];
    }
  }
}

// In place: a block takes 16 / parts columns of 16 bytes of K or of V of one kv head, and the first such block the weights.
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const EvictParams p) {
  const int b = static_cast<int>(blockIdx.y), hkv = p.a.hkv;
  int x = static_cast<int>(blockIdx.x);
  const int part = x % p.parts;
  x /= p.parts;
  const bool is_v = (x & 1) != 0;
  const int hk = x >> 1;
  const int lanes = 16 / p.parts, rows = kMoveThreads / lanes;  // threads to a row; rows at once
  const int column = part * lanes + static_cast<int>(threadIdx.x) % lanes, row = static_cast<int>(threadIdx.x) / lanes;
  const bool weighs = !is_v && column == 0;
  uint16_t* cache = static_cast<uint16_t*>(is_v ? p.a.v_cache : p.a.k_cache);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = length_of(p, b, false);
  if (n <= p.a.budget) return;
  const int32_t* kept = p.a.kept + (static_cast<int64_t>(b) * hkv + hk) * p.a.budget;
  int64_t to[kAhead], w_to[kAhead], next_to[kAhead], next_w_to[kAhead];
  uint4 d[kAhead], next_d[kAhead];
  float w[kAhead], next_w[kAhead];
  auto read = [&](int j0, int64_t (&to_)[kAhead], int64_t (&w_to_)[kAhead], uint4 (&d_)[kAhead], float (&w_)[kAhead]) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = j0 + i * rows + row;
      to_[i] = -1;
      if (j < p.a.budget) {
        const int t = kept[j];
        if (t != j) {  // else it is there already
          const int from = block_of(p, p.a.block_tables, p.a.bt_stride, b, t);
          const int dest = block_of(p, p.a.block_tables, p.a.bt_stride, b, j);
          if (from >= 0 && dest >= 0) {
            d_[i] = ld_row(cache + ((static_cast<int64_t>(from) * kBlockSize + t % kBlockSize) * hkv + hk) * kHeadDim +
                           column * 8);
            if (weighs) w_[i] = p.a.weights[weight_place(p, from, hk, t)];
            to_[i] = ((static_cast<int64_t>(dest) * kBlockSize + j % kBlockSize) * hkv + hk) * kHeadDim + column * 8;
            w_to_[i] = weight_place(p, dest, hk, j);
          }
        }
      }
    }
  };
  const int chunk = rows * kAhead;
  read(0, to, w_to, d, w);
  for (int j0 = 0; j0 < p.a.budget; j0 += chunk) {
    if (j0 + chunk < p.a.budget) read(j0 + chunk, next_to, next_w_to, next_d, next_w);
    __syncthreads();  // the whole chunk has been read before any of it is written
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (to[i] >= 0) {
        *reinterpret_cast<uint4*>(cache + to[i]) = d[i];
        if (weighs) p.a.weights[w_to[i]] = w[i];
      }
      to[i] = next_to[i];
      w_to[i] = next_w_to[i];
      d[i] = next_d[i];
      w[i] = next_w[i];
    }
  }
}

template <typename... Args>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int kThreads>
cudaError_t launch_select(const EvictParams& p, cudaStream_t stream) {
  // the attribute holds for the current device; setting it again costs the host less than a launch
  const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<kThreads>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (3 * kBins + kCached) * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.a.hkv * p.ranks), static_cast<unsigned>(p.a.num_seqs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>((p.ranks > 1 ? 3 : 1) * kBins + p.cached) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(p.ranks);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<kThreads>, p);
}

cudaError_t launch_evict(const EvictArgs& a, unsigned int* err, cudaStream_t stream) {
  EvictParams p{};
  p.a = a;
  p.err = err;
  // Few (sequence, kv head) pairs with many tokens each: up to 8 blocks share one, of 1024 threads. Many pairs: smaller
  // blocks, several to an SM, hide one another's waits.
  const int64_t blocks = static_cast<int64_t>(a.num_seqs) * a.hkv;
  p.ranks = 1;
  while (p.ranks < kMaxRanks && blocks * p.ranks * 2 <= 2 * 152 && a.max_ctx >= 2048 * p.ranks) p.ranks *= 2;
  const int share = (a.max_ctx + p.ranks - 1) / p.ranks;
  p.cached = share < kCached ? share : kCached;
  const cudaError_t e =
      blocks * p.ranks <= 2 * 152 || share > 16384 ? launch_select<1024>(p, stream) : launch_select<256>(p, stream);
  if (e != cudaSuccess) return e;
  if (a.new_tables) {
    const int64_t most = static_cast<int64_t>(a.budget < a.max_ctx ? a.budget : a.max_ctx) * a.hkv;
    const int64_t per = kHalfWarps * kAhead * kRounds;
    const dim3 grid(static_cast<unsigned>((most + per - 1) / per), static_cast<unsigned>(a.num_seqs));
    return most > 0 ? launch_behind(evict_copy_kernel, grid, kMoveThreads, stream, p) : cudaSuccess;
  }
  // columns of a row are shared out until there are blocks for every SM (32 bytes, a sector, at least)
  p.parts = 1;
  while (p.parts < 8 && blocks * 2 * p.parts < 2 * 152) p.parts *= 2;
  const dim3 grid(static_cast<unsigned>(a.hkv * 2 * p.parts), static_cast<unsigned>(a.num_seqs));
  return launch_behind(evict_compact_kernel, grid, kMoveThreads, stream, p);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pkv

extern "C" int pkv_evict_kvcache(void* k_cache, void* v_cache, float* weights, int32_t num_blocks,
                                 const int32_t* block_tables, int32_t block_table_stride, const int32_t* context_lens,
                                 int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                 int32_t max_context_len, int32_t budget, int32_t first, int32_t recent,
                                 const int32_t* new_block_tables, int32_t new_block_table_stride, int32_t* kept,
                                 int32_t* new_context_lens, cudaStream_t stream) {
  if (head_dim != pkv::kHeadDim || block_size != pkv::kBlockSize || num_kv_heads <= 0 || num_kv_heads > 8192)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs < 0 || num_seqs > 65535 || num_blocks < 0 || block_table_stride < 0 || max_context_len < 0 ||
      max_context_len > (1 << 24) || budget < 1 || budget > (1 << 24) || first < 0 || recent < 0 ||
      first > budget || recent > budget - first)
    return PKV_ERR_BAD_SIZE;
  if (num_seqs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !weights || !block_tables || !context_lens || !kept || !new_context_lens)
    return PKV_ERR_NULL_POINTER;
  const int32_t most = budget < max_context_len ? budget : max_context_len;
  if (new_block_tables && static_cast<int64_t>(new_block_table_stride) * block_size < most) return PKV_ERR_BAD_SIZE;
  if (!pkv::aligned(k_cache, 16) || !pkv::aligned(v_cache, 16)) return PKV_ERR_ALIGNMENT;
  for (const void* p : {static_cast<const void*>(weights), static_cast<const void*>(block_tables),
                        static_cast<const void*>(context_lens), static_cast<const void*>(new_block_tables),
                        static_cast<const void*>(kept), static_cast<const void*>(new_context_lens)})
    if (!pkv::aligned(p, 4)) return PKV_ERR_ALIGNMENT;
  // the new lengths are written while the old ones are still read
  const intptr_t apart = reinterpret_cast<intptr_t>(new_context_lens) - reinterpret_cast<intptr_t>(context_lens);
  if (apart < 4 * static_cast<intptr_t>(num_seqs) && -apart < 4 * static_cast<intptr_t>(num_seqs)) return PKV_ERR_BAD_SIZE;
  unsigned int* err = nullptr;
  const int st = pkv::device_error_word(&err);
  if (st != PKV_OK) return st;
  const pkv::EvictArgs a{k_cache,      v_cache,   weights,      num_blocks,      block_tables,
                         block_table_stride, context_lens, num_seqs, num_kv_heads, max_context_len,
                         budget,       first,     recent,       new_block_tables, new_block_table_stride,
                         kept,         new_context_lens};
  if (pkv::launch_evict(a, err, stream) == cudaSuccess) return PKV_OK;
  (void)cudaGetLastError();
  return PKV_ERR_CUDA;
}
