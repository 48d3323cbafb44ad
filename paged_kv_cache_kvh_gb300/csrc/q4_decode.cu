// q4_decode.cu -- single-query attention over the 4-bit paged cache (split-KV).
//
// For sequence b, query head h and kv head h / G, with c, s, z the codes,
// scales and minima of q4.cuh (group g of 32 dims):
//   logit_t = scale * sum_g (s_tg * sum_{d in g} q_d c_td + z_tg * sum_{d in g} q_d)
//   out_d   = sum_t p_t (s_tg c_td + z_tg) / sum_t p_t,  p = softmax(logit)
// The codes are used exactly as stored; no 16-bit K or V row is ever formed.
//
// What bounds it: 160 bytes per (token, kv head) from HBM, which at the copy
// rate are 47 codes a clock and SM. Widening and multiplying them on the CUDA
// cores (an unpack and two multiply-adds per code and query head) would need more
// issue slots than an SM has, so both products run on mma.sync m16n8k16:
//  * A holds 16 tokens x 16 dims of codes (K) or 16 dims x 16 tokens (V) as
//    fp16. A code in the low nibble of each 16-bit half, w & 0x000f000f, is
//    already an fp16 number: the subnormal code * 2^-24, exactly; the next
//    nibble, w & 0x00f000f0, is 16 times that. So 8 codes cost four ANDs and
//    a shift, and the powers of two are taken out of q, p and the result.
//  * B's 8 columns are 2 query heads x 4 groups (column 2 g + h). For K, column
//    2 g + h holds head h's q in the dims of group g and 0 elsewhere, so one
//    accumulator ends with every group's own sum: lane (r, t) of the C fragment
//    has tokens r, r + 8, group t, both heads. For V, column 2 g + h holds
//    p_t s_tg: C columns of other groups than the row's dims are not used.
//  * The sum over the groups, four lanes, is a tf32 product with ones (each
//    addend as a high and a low part, 2^-22 of it at most is lost), and
//    z_tg . sum q is another, whose C starts at minus the running maximum:
//    the logits come out relative to it. Shuffles instead took 184 us where
//    these took 163.
//  * V's 16-bit fields are transposed by the load from shared memory (ldmatrix),
//    p goes from C's layout to B's by movmatrix (8 x 8 transposes in registers).
//  * q is scaled by a power of two per head so that fp16 holds it exactly
//    (elements below 2^-38 of the head's largest are rounded); p s is scaled by
//    a running power of two and rounded to fp16 (relative 2^-11, as p is in any
//    tensor-core product; kCentred below). Sums, maxima and the z terms stay in fp32.
//
// Work: an item is a chunk of one sequence for a pair of query heads that share a
// kv head (for a single head where each has its own; with four or more to a kv
// head the pairs run next to one another and read the tiles from L2). A warp works
// through items alone, 64 tokens a step: bulk copies (K and V tiles of one (block,
// head) are contiguous) fetch K two steps ahead and V one step ahead into its own
// 15 KB of shared memory, and it waits on its own barriers, so no warp ever waits
// for another. One CTA of 12 warps per SM. Chunks: chunk_tokens. Every CTA derives
// the item table from context_lens: whole chunks first, then the sequences' short
// last chunks, longest first. Warp w starts on item w and takes the next ones from
// a counter in the workspace, asked two steps before its item ends.
// Partial results (m, l, o) of sequences with several chunks go to the workspace;
// the ticket is taken a step later, when the writes have landed, and the warp that
// takes the last one merges them (no waiting): up to 16 chunks at once, groups of
// 16 and then the groups beyond that.
// The fused step quantises a sequence's new row in the warps that read its last
// tile, which put it over what was fetched; one of them writes it to the cache.
//
// Measured: 256 sequences of 512..4096 tokens, 16 query heads on 8: 139 us,
// 5.5 TB/s (81 % of the copy rate); 512 of 800 on average, fp16: 101 us, 76 %; one of
// 40007, 32 on 8: 31 us. With every block table folded onto a few blocks that
// stay in L2 the first takes the same time: it is bound by execution, about 512
// warp instructions per 32 tokens and pair of heads at 0.48 a clock and scheduler.
// Measured and not kept: 16 warps of 32-token steps (165 us: more control per
// token), 8 warps (163), one K buffer and 16 warps (141), accumulators rescaled
// without a branch (154), other orders of the products (150 as they stood then),
// shifts as multiplications (166), bf16 queries as two e4m3 parts against codes that
// are e4m3 numbers as they stand (183: fewer instructions, but spills and longer
// chains).
#include <atomic>
#include <type_traits>

#include "q4.cuh"

namespace pkv {

struct FusedStore {
  const void* k;
  int64_t k_row_stride;
  const void* v;
  int64_t v_row_stride;
  const int32_t* slot_mapping;
};

namespace {

constexpr int kUnit = 64;                                    // tokens per stage
constexpr int kHalfUnit = 32;                                // the shortest chunk
constexpr int kUnitTiles = kUnit / kQ4Tile;
constexpr int kUnitBytes = kUnitTiles * kQ4TileBytes;        // 5120, of K and of V each
constexpr int kMaxChunk = 32;                                // units per chunk at most
constexpr int kMaxSeqs = 768;                                // sequences per launch (item table in shared memory)
constexpr int kClasses = 8;                                  // sizes that short chunks are sorted into
constexpr int kFan = 16;                                     // chunks merged at once
constexpr int kFirst = 1 << 8, kLast = 1 << 9, kNew = 1 << 10;  // a unit's flags: first and last of its item, holds a new row
constexpr int kSpoilt = INT32_MIN;                           // see the end of the kernel
constexpr uint32_t kTf32Mask = 0xffffe000u;                  // the bits that a tf32 operand keeps
constexpr uint32_t kOne = 0x3f800000u;                       // 1.0f

constexpr int kWarps = 12;                                   // per CTA; one CTA per SM
constexpr int kThreads = kWarps * 32;

// A warp's shared memory: two units of K, one of V, the query rows of two items
// (they arrive with an item's first K), and what its lanes share about them.
struct WarpInfo {
  int4 item[4];       // {sequence, head, chunk | chunks of the sequence << 16, -} of the items under way
  int64_t place[2];   // per K slot: where the unit starts in the caches
  int32_t unit[2];    // tokens, flags
  uint32_t bytes[2];  // to fetch of K and of V each
  uint64_t bars[3];   // K, K, V arrived
};

struct Q4DecodeParams {
  const uint16_t* q;
  int64_t q_row_stride;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  int32_t num_blocks;
  int32_t hkv;
  int32_t rows;   // items per (sequence, chunk): pairs of query heads that share a kv head, or single ones
  int32_t share;  // rows per kv head
  const int32_t* block_tables;
  int32_t bt_stride;
  const int32_t* context_lens;
  int32_t max_ctx;
  int32_t num_seqs;
  float scale_log2;
  uint16_t* out;
  int32_t* work;     // {next item, warps done}, zero between calls; kSpoilt in the latter after a wait that ran out
  int32_t* tickets;  // one per slot, zero between calls
  float2* ml;        // [slot][G] (max in log2 units, sum)
  float* opart;      // [slot][G][128], not normalised; slot (whole chunks before b + b + chunk) * hkv + head
  int64_t max_slots;
  // the step's new rows (pkv_store_decode_q4); k_new == nullptr for plain decode
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t k_new_stride;
  int64_t v_new_stride;
  const int32_t* slot_mapping;
  uint8_t* k_cache_w;
  uint8_t* v_cache_w;
  unsigned int* err;
};

// Tokens per chunk. Where half units suffice for one chunk to a warp, chunks of
// 32 tokens (a short call is bound by the time of one chunk). Otherwise whole
// units: x is the number that each warp would get; up to kMaxChunk, one chunk
// each; beyond, as many rounds of equal chunks as keep a chunk within kMaxChunk.
__host__ __device__ inline int chunk_tokens(int64_t half_units, int64_t units) {
  constexpr int64_t plan = int64_t{152} * kWarps;
  if (half_units <= plan) return kHalfUnit;
  const int64_t x = (units + plan - 1) / plan;
  const int64_t rounds = (x + kMaxChunk - 1) / kMaxChunk;
  return static_cast<int>((x + rounds - 1) / rounds) * kUnit;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
  return r;
}
// Four 8 x 8 matrices of 16-bit fields, transposed: lane i gives the address of
// row i % 8 of matrix i / 8; lane (r, t) gets column r of rows 2t, 2t + 1.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&d)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
               : "r"(addr));
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the first of a chain: C = 0
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D = A B + C with C left as it is, and in place
__device__ __forceinline__ void mma1688_tf32_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma1688_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Whole-warp bounded wait, after a first test has failed.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, unsigned int* err) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    for (int i = 0; i < 64; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs)) {
      flag_error(err, PKV_DEVERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// the power of two 2^e, e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127; }

// Merges n partials (slots first, first + stride, ...) of all G query heads, 4
// dims per lane: o = sum 2^(m - M) o_i, l = sum 2^(m - M) l_i, M the largest m.
// The partials sit in L2: the loads of kAhead slots and every head are in flight
// together.
template <int G>
__device__ __forceinline__ void merge_slots(const Q4DecodeParams& p, int64_t first, int64_t stride, int n, int lane,
                                            float (&M)[G], float (&den)[G], float4 (&acc)[G]) {
  constexpr int kAhead = G == 1 ? 8 : 4;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    M[h] = -INFINITY;
    den[h] = 0.f;
    acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 1
  for (int c0 = 0; c0 < n; c0 += kAhead) {
    float2 ml[kAhead][G];
    float4 o[kAhead][G];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t slot = (first + min(c0 + i, n - 1) * stride) * G;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        ml[i][h] = __ldcg(p.ml + slot + h);
        o[i][h] = __ldcg(reinterpret_cast<const float4*>(p.opart + (slot + h) * kHeadDim) + lane);
        if (c0 + i >= n) ml[i][h].x = -INFINITY;  // the last one again: no weight
      }
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float Mg = M[h];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) Mg = fmaxf(Mg, ml[i][h].x);
      const float Mu = (Mg == -INFINITY) ? 0.f : Mg;
      const float sc = ex2_approx(M[h] - Mu);
      M[h] = Mg;
      den[h] *= sc;
      acc[h].x *= sc;
      acc[h].y *= sc;
      acc[h].z *= sc;
      acc[h].w *= sc;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const bool there = c0 + i < n;  // 0 * NaN must not be added
        const float w = ex2_approx(ml[i][h].x - Mu);
        den[h] = there ? fmaf(w, ml[i][h].y, den[h]) : den[h];
        acc[h].x = there ? fmaf(w, o[i][h].x, acc[h].x) : acc[h].x;
        acc[h].y = there ? fmaf(w, o[i][h].y, acc[h].y) : acc[h].y;
        acc[h].z = there ? fmaf(w, o[i][h].z, acc[h].z) : acc[h].z;
        acc[h].w = there ? fmaf(w, o[i][h].w, acc[h].w) : acc[h].w;
      }
    }
  }
}

template <Elem E, int G>
__global__ void __launch_bounds__(kThreads, 1) q4_decode_kernel(const Q4DecodeParams p) {
  using Ops = ElemOps<E>;
  // What rounding p s to fp16 loses comes back multiplied by the code. With codes
  // taken from their middle, c - 7.5, that is half as much: z + 7.5 s takes z's
  // place, and 7.5 times the sum of the rounded p s (a product with ones) is taken
  // off at the end. For bf16 the result's own rounding is 8 times larger than
  // either, so only fp16 pays for it: 512 sequences of 800 tokens on average take
  // 101 us instead of 98, at an error of 0.00025 instead of 0.00038 (the result's
  // rounding alone: 0.0002).
  constexpr bool kCentred = E == Elem::kF16;
  constexpr int kQBytes = G * kHeadDim * 2;   // one item's query rows
  constexpr int kWarpBytes = 3 * kUnitBytes + 2 * kQBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  WarpInfo* info_all = reinterpret_cast<WarpInfo*>(smem + kWarps * kWarpBytes);
  int* sF = reinterpret_cast<int*>(info_all + kWarps);  // [num_seqs + 1] whole chunks before b
  int* sCtx = sF + kMaxSeqs + 1;                                                   // [num_seqs]
  int* plist = sCtx + kMaxSeqs;                                                    // sequences with a short last chunk
  int* red = plist + kMaxSeqs;                                                     // [2][kWarps], then [9][32]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.num_seqs;
  const int n_ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const bool spoilt = __ldcg(p.work + 1) < 0;  // (on its way together with the lengths)

  // ---- item table (every CTA builds the same one) ----
  // Whole chunks first, in sequence order, then the short last chunks in kClasses
  // sizes, longest first: the items that end the call are the shortest. A warp
  // holds sequences i * kThreads + tid, 32 consecutive ones (a group) at a time.
  int chunk, n_full, n_part = 0;
  if (B <= 32) {
    // One sequence per lane, every warp for itself (the sizes stay in registers,
    // warp 0 writes the table). Short chunks follow in sequence order.
    int ctx = 0;
    if (lane < B) {
      ctx = p.context_lens[lane];
      if (ctx < 0 || ctx > p.max_ctx || ctx > static_cast<int64_t>(p.bt_stride) * kBlockSize) {
        if (cta == 0 && warp == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
        ctx = 0;
      }
    }
    if (lane < 3) mbar_init(smem_u32(info_all[warp].bars + lane), 1);
    mbar_fence_init();
    int halves = (ctx + kHalfUnit - 1) / kHalfUnit, units = (ctx + kUnit - 1) / kUnit;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      halves += __shfl_xor_sync(0xffffffffu, halves, off);
      units += __shfl_xor_sync(0xffffffffu, units, off);
    }
    chunk = chunk_tokens(static_cast<int64_t>(halves) * p.rows, static_cast<int64_t>(units) * p.rows);
    const int full = static_cast<int>(static_cast<unsigned>(ctx) / static_cast<unsigned>(chunk));
    int scan = full;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, off);
      if (lane >= off) scan += y;
    }
    n_full = __shfl_sync(0xffffffffu, scan, 31);
    const uint32_t part = __ballot_sync(0xffffffffu, full * chunk < ctx);
    n_part = __popc(part);
    if (warp == 0) {
      if (lane < B) {
        sCtx[lane] = ctx;
        sF[lane] = scan - full;
        if (full * chunk < ctx) plist[__popc(part & ((1u << lane) - 1u))] = lane;
      }
      if (lane == 0) sF[B] = n_full;
    }
    __syncthreads();
  } else {
    constexpr int kPer = (kMaxSeqs + kThreads - 1) / kThreads;
    static_assert(kPer * kWarps <= 32, "one lane per group below");
    int ctx[kPer];
    int halves = 0, units = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = i * kThreads + tid;
      ctx[i] = 0;
      if (b < B) {
        const int c = p.context_lens[b];
        if (c < 0 || c > p.max_ctx || c > static_cast<int64_t>(p.bt_stride) * kBlockSize) {
          if (cta == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
        } else {
          ctx[i] = c;
        }
        sCtx[b] = ctx[i];
      }
      halves += (ctx[i] + kHalfUnit - 1) / kHalfUnit;
      units += (ctx[i] + kUnit - 1) / kUnit;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      halves += __shfl_xor_sync(0xffffffffu, halves, off);
      units += __shfl_xor_sync(0xffffffffu, units, off);
    }
    if (lane == 0) {
      red[warp] = halves;
      red[kWarps + warp] = units;
    }
    if (lane < 3) mbar_init(smem_u32(info_all[warp].bars + lane), 1);
    mbar_fence_init();
    __syncthreads();
    int64_t all_halves = 0, all_units = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      all_halves += red[w];
      all_units += red[kWarps + w];
    }
    chunk = chunk_tokens(all_halves * p.rows, all_units * p.rows);
    __syncthreads();  // red is written again
    int full[kPer], cls[kPer], scan[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      full[i] = static_cast<int>(static_cast<unsigned>(ctx[i]) / static_cast<unsigned>(chunk));
      const int rest = ctx[i] - full[i] * chunk;
      cls[i] = rest > 0 ? kClasses - 1 - (rest * kClasses - 1) / chunk : -1;
      scan[i] = full[i];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, scan[i], off);
        if (lane >= off) scan[i] += y;
      }
      int mine = 0;
#pragma unroll
      for (int k = 0; k < kClasses; ++k) {
        const int c = __popc(__ballot_sync(0xffffffffu, cls[i] == k));
        if (lane == k) mine = c;
      }
      const int group = i * kWarps + warp;
      if (lane < kClasses) red[lane * 32 + group] = mine;
      if (lane == 31) red[kClasses * 32 + group] = scan[i];
    }
    __syncthreads();
    // lane = group: what comes before each group
    constexpr int kGroups = kPer * kWarps;
    int before[kClasses + 1];
#pragma unroll
    for (int k = 0; k <= kClasses; ++k) {
      const int own = lane < kGroups ? red[k * 32 + lane] : 0;
      int x = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      const int total = __shfl_sync(0xffffffffu, x, 31);
      before[k] = x - own + (k < kClasses ? n_part : 0);
      if (k < kClasses)
        n_part += total;
      else
        n_full = total;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = i * kThreads + tid, group = i * kWarps + warp;
      const int f0 = __shfl_sync(0xffffffffu, before[kClasses], group);
      if (b < B) sF[b] = f0 + scan[i] - full[i];
#pragma unroll
      for (int k = 0; k < kClasses; ++k) {
        const uint32_t same = __ballot_sync(0xffffffffu, cls[i] == k);
        const int at = __shfl_sync(0xffffffffu, before[k], group);
        if (cls[i] == k) plist[at + __popc(same & ((1u << lane) - 1u))] = b;
      }
    }
    if (tid == 0) sF[B] = n_full;
    __syncthreads();
  }
  if (spoilt) {
    if (tid == 0 && cta == 0) flag_error(p.err, PKV_DEVERR_TIMEOUT);
    return;
  }
  const int64_t n_items = static_cast<int64_t>(n_full + n_part) * p.rows;
  if (static_cast<int64_t>(n_full + B) * p.rows > p.max_slots) {  // cannot happen: the workspace bound covers every table
    if (tid == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
    return;
  }

  // rows without context: zeros, and nothing to store
  for (int b = cta * kWarps + warp; b < B; b += n_ctas * kWarps) {
    if (sCtx[b] == 0) {
      uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(b) * p.rows * G * kHeadDim);
      for (int i = lane; i < p.rows * G * (kHeadDim / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
      if (p.k_new != nullptr && lane == 0 && p.slot_mapping[b] != -1) flag_error(p.err, PKV_DEVERR_BAD_SLOT);
    }
  }

  const uint32_t k_buf = smem_u32(smem) + warp * kWarpBytes, v_buf = k_buf + 2 * kUnitBytes;
  const uint32_t q_buf = v_buf + kUnitBytes;
  WarpInfo* info = info_all + warp;
  const uint32_t k_full = smem_u32(info->bars), v_full = k_full + 16;
  const int r = lane >> 2, t = lane & 3;
  const int W = n_ctas * kWarps;
  const bool dynamic = n_items > W;

  // ---- the issuing side: which unit is fetched next ----
  int64_t item = static_cast<int64_t>(warp) * n_ctas + cta;
  // Lane 0 asks the counter for the next item two units before this one ends: early
  // enough to hide the answer's way, late enough to leave the last items to the
  // warps that get to them first.
  int next_raw = 0;
  bool asked = false;
  auto ask = [&]() {
    if (lane == 0) next_raw = atomicAdd(p.work, 1);
    asked = true;
  };
  int ib = 0, ihead = 0, itok = 0;     // sequence, head, next token
  int left = 0;                        // tokens of the chunk not asked for yet; 0: no more work
  int items = 0;                       // items resolved
  bool ifirst = false, itail = false;  // next unit is an item's first; the item is its sequence's last chunk
  int ipb = -1;                        // block of the unit to fetch; read one unit ahead of its use
  bool fresh = false;                  // ipb has not been checked and turned into ioff yet
  int64_t ioff = -1;                   // where the next unit starts in the caches; -1: a bad block
  auto look_up = [&]() {
    ipb = p.block_tables[static_cast<int64_t>(ib) * p.bt_stride + itok / kBlockSize];
    fresh = true;
  };
  auto resolve = [&]() {  // item -> sequence, chunk, head (whole warp)
    const int ci = static_cast<int>(static_cast<unsigned>(item) / static_cast<unsigned>(p.rows));
    ihead = static_cast<int>(item) - ci * p.rows;
    int c;
    if (ci < n_full) {
      // largest b with sF[b] <= ci, 32 probes at a time
      const int step = (B + 31) / 32;
      const int probe = lane * step;
      const int hi = __popc(__ballot_sync(0xffffffffu, probe < B && sF[probe] <= ci)) - 1;
      const int probe2 = hi * step + lane;
      const int cnt = __popc(__ballot_sync(0xffffffffu, lane < step && probe2 < B && sF[probe2] <= ci));
      ib = hi * step + cnt - 1;
      c = ci - sF[ib];
    } else {
      ib = plist[ci - n_full];
      c = sF[ib + 1] - sF[ib];
    }
    const int ctx = sCtx[ib];
    int nch = sF[ib + 1] - sF[ib];
    nch += nch * chunk < ctx ? 1 : 0;
    itok = c * chunk;
    left = min(chunk, ctx - itok);
    ifirst = true;
    itail = c == nch - 1;
    if (lane == 0) info->item[items & 3] = make_int4(ib, ihead, c | (nch << 16), 0);
    ++items;
    look_up();
  };
  if (item < n_items) resolve();
  int issued = 0;  // units whose K has been asked for
  auto issue_k = [&]() {  // fetches the next unit's K (whole warp)
    if (left <= 0) return;
    if (fresh) {
      fresh = false;
      ioff = -1;
      if (ipb >= 0 && ipb < p.num_blocks)
        ioff = (static_cast<int64_t>(ipb) * p.hkv + ihead / p.share) * kQ4RecordBytes + (itok % kBlockSize) / kQ4Tile * kQ4TileBytes;
      else if (lane == 0)
        flag_error(p.err, PKV_DEVERR_BAD_BLOCK);
    }
    const int ntok = min(kUnit, left);
    const bool last = left <= kUnit;
    int flags = ntok | (ifirst ? kFirst : 0) | (last ? kLast : 0);
    if (p.k_new != nullptr && last && itail) {
      // the unit holds the newest position: the computing side puts its row in
      const int64_t slot = p.slot_mapping[ib];
      if (slot != -1) {
        if (ioff >= 0 && slot == static_cast<int64_t>(ipb) * kBlockSize + (itok + ntok - 1) % kBlockSize)
          flags |= kNew;
        else if (lane == 0 && ihead == 0)
          flag_error(p.err, PKV_DEVERR_BAD_SLOT);
      }
    }
    const uint32_t bytes = ioff < 0 ? 0u : static_cast<uint32_t>((ntok + kQ4Tile - 1) / kQ4Tile) * kQ4TileBytes;
    if (lane == 0) {
      const int s = issued & 1;
      info->unit[s] = ioff < 0 ? flags & ~0xff : flags;
      info->place[s] = ioff;
      info->bytes[s] = bytes;
      mbar_arrive_expect_tx(k_full + 8 * s, bytes + (ifirst ? kQBytes : 0));
      if (bytes > 0) bulk_g2s(k_buf + s * kUnitBytes, p.k_cache + ioff, bytes, k_full + 8 * s);
      if (ifirst)
        bulk_g2s(q_buf + s * kQBytes, p.q + static_cast<int64_t>(ib) * p.q_row_stride + ihead * G * kHeadDim, kQBytes,
                 k_full + 8 * s);
    }
    ifirst = false;
    ++issued;
    itok += kUnit;
    left -= kUnit;
    if (last) {
      left = 0;
      if (dynamic) {
        if (!asked) ask();
        asked = false;
        item = static_cast<int64_t>(W) + __shfl_sync(0xffffffffu, next_raw, 0);
        if (item < n_items) resolve();
      }
    } else {
      if (dynamic && !asked && left <= 2 * kUnit) ask();
      if (itok % kBlockSize == 0)
        look_up();
      else if (ioff >= 0)
        ioff += kUnitBytes;
    }
  };
  auto issue_v = [&](int n) {  // fetches V of unit n, whose K has been asked for
    if (n < issued && lane == 0) {
      const uint32_t bytes = info->bytes[n & 1];
      mbar_arrive_expect_tx(v_full, bytes);
      if (bytes > 0) bulk_g2s(v_buf, p.v_cache + info->place[n & 1], bytes, v_full);
    }
  };
  issue_k();
  issue_v(0);
  issue_k();

  // ---- the computing side ----
  // Lane (r, t): K rows (and C rows) of tokens r, r + 8, group t. For V, lane i of
  // a 4-matrix transposing load addresses 16-byte chunk i / 8 of token i % 8; lane
  // (r, t) then holds, of tokens 2t, 2t + 1, four dims of group r & 3 per chunk.
  const uint32_t par_off = kQ4TileParams + r * kQ4ParamBytes + t * 4;
  const uint32_t v_off = (lane & 7) * kQ4CodeBytes + (((lane >> 3) ^ ((lane & 4) >> 1)) << 4);
  uint32_t qb[8][2];         // B fragments of q, one per 16 dims
  uint32_t qs_b[G][2];       // B fragment of sum q over group t: high and low part
  float kc[2];               // per head: the power of two taken out of q and the codes, times scale * log2(e)
  float acc[8][4];
  float ones[4];             // kCentred: sum of the rounded p s, group t
  uint64_t l2[G], z2[G];     // sums of p and of p z (kCentred: p (z + 7.5 s)), tokens r and r + 8 apart
  float m[G];                // running maximum, -INFINITY before the first unit
  float from[G][4];          // minus the maximum that logits are taken relative to (a C fragment)
  float nu = 1.f;

  int done = 0;              // units worked through
  int items_done = 0;
  bool pending = false;      // a partial result is written, its ticket not taken yet
  int pend_b = 0, pend_head = 0, pend_c = 0;  // pend_c: chunk | chunks << 16
  while (true) {
    const bool have = done < issued;
    int flags = 0;
    if (have) {
      const int s = done & 1;
      const uint32_t k_phase = (done >> 1) & 1;
      if (!__all_sync(0xffffffffu, mbar_try_wait(k_full + 8 * s, k_phase)) && !wait_warp(k_full + 8 * s, k_phase, p.err))
        break;
      const uint32_t kst = k_buf + s * kUnitBytes;
      flags = info->unit[s];
      const int ntok = flags & 0xff;
      uint32_t new_codes = 0, new_par = 0;
      if (flags & kNew) {
        // The step's new row: lanes 0..15 quantise K's, lanes 16..31 V's, 8 dims
        // each, and write it to the cache and over what was fetched of it.
        const int4 it = info->item[items_done & 3];
        const int lane16 = lane & 15, j = lane16 >> 2, tt = lane16 & 3, tok = (ntok - 1) % kQ4Tile;
        const bool is_v = lane >= 16;
        const uint16_t* src = (is_v ? p.v_new + it.x * p.v_new_stride : p.k_new + it.x * p.k_new_stride) +
                              it.y / p.share * kHeadDim + lane16 * 8;
        new_codes = quantise8<E>(*reinterpret_cast<const uint4*>(src), new_par);
        const uint32_t vcodes = v_exchange(new_codes, j);
        if (is_v) new_codes = vcodes;
        const int word = is_v ? q4_v_word(tok, j, tt) : q4_k_word(tok, j, tt);
        const int tile = (ntok - 1) / kQ4Tile * kQ4TileBytes;
        uint8_t* dst = (is_v ? p.v_cache_w : p.k_cache_w) + info->place[s] + tile;
        if (it.y % p.share == 0) {  // one of the items that share the kv head
          *reinterpret_cast<uint32_t*>(dst + word) = new_codes;
          if (tt == 0) *reinterpret_cast<uint32_t*>(dst + q4_param(tok, j)) = new_par;
        }
        if (!is_v) {
          sts32(kst + tile + word, new_codes);
          if (tt == 0) sts32(kst + tile + q4_param(tok, j), new_par);
        }
        fence_proxy_async_smem();  // the stage's next copy comes after these stores
        __syncwarp();
      }
      if (flags & kFirst) {
        // ---- a new item: query fragments ----
        {
          const int h = r & 1;  // the column's head; its group is r >> 1
          uint4 raw = make_uint4(0, 0, 0, 0);
          if (h < G) raw = lds128(q_buf + s * kQBytes + h * kHeadDim * 2 + ((r >> 1) * 32 + t * 8) * 2);
          float x[8] = {Ops::lo(raw.x), Ops::hi(raw.x), Ops::lo(raw.y), Ops::hi(raw.y),
                        Ops::lo(raw.z), Ops::hi(raw.z), Ops::lo(raw.w), Ops::hi(raw.w)};
          float big = 0.f, sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[i]));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 8));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 16));
          const int e = big > 0.f ? 13 - exponent_of(big) : 0;  // the largest |q| goes to [2^13, 2^14)
          const float f = pow2(min(e, 120));
          // From |q| = 2^114 on, 2^24 / f would pass fp32: logits are then taken as
          // if q were smaller. Their steps are still far above 1 (s >= 2^-24), so
          // the largest one takes all the weight either way.
          const float least = pow2(-100);
          const float shrink = fminf(f * pow2(100), 1.f);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(x[i], shrink, sum);
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          const float f16 = f * 0.0625f;  // for the codes that A holds 16 times too large
          const uint32_t own[4] = {pack_f16(x[0] * f, x[4] * f), pack_f16(x[1] * f16, x[5] * f16),
                                   pack_f16(x[2] * f, x[6] * f), pack_f16(x[3] * f16, x[7] * f16)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // group j's two fragments: 0 outside the column's own group
            const bool on = j == (r >> 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) qb[2 * j + i / 2][i & 1] = on ? own[i] : 0u;
          }
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            const float fh = __shfl_sync(0xffffffffu, f, 4 * h2);
            kc[h2] = __fdividef(16777216.f, fmaxf(fh, least)) * p.scale_log2;
            const float qs = __shfl_sync(0xffffffffu, sum, (2 * t + h2) * 4) * p.scale_log2;
            if (h2 < G) {
              qs_b[h2 % G][0] = __float_as_uint(qs) & kTf32Mask;
              qs_b[h2 % G][1] = __float_as_uint(qs - __uint_as_float(__float_as_uint(qs) & kTf32Mask));
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
          if (kCentred) ones[0] = ones[1] = ones[2] = ones[3] = 0.f;
        }
#pragma unroll
        for (int h = 0; h < G; ++h) {
          m[h] = -INFINITY;
          from[h][0] = from[h][1] = from[h][2] = from[h][3] = 0.f;
          l2[h] = z2[h] = 0;
        }
        nu = 1.f;
      }

      // ---- logits, less the running maximum: lg[h][tile][half], tokens r + 8 half ----
      float lg[G][kUnitTiles][2];
#pragma unroll
      for (int pair = 0; pair < kUnitTiles / 2; ++pair) {
        if (pair * kHalfUnit >= ntok) {
#pragma unroll
          for (int h = 0; h < G; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) lg[h][2 * pair + i / 2][i & 1] = -INFINITY;
          continue;
        }
        float c[2][4];
        uint4 w0[2], w1[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t base = kst + (2 * pair + i) * kQ4TileBytes + lane * 16;
          w0[i] = lds128(base);
          w1[i] = lds128(base + 8 * kQ4CodeBytes);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a = j == 0 ? w0[i].x : j == 1 ? w0[i].y : j == 2 ? w0[i].z : w0[i].w;
            const uint32_t b = j == 0 ? w1[i].x : j == 1 ? w1[i].y : j == 2 ? w1[i].z : w1[i].w;
            const uint32_t ah = a >> 8, bh = b >> 8;
            if (j == 0)
              mma16816_first(c[i], a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u, qb[0][0],
                             qb[0][1]);
            else
              mma16816(c[i], a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u, qb[2 * j][0],
                       qb[2 * j][1]);
            mma16816(c[i], ah & 0x000f000fu, bh & 0x000f000fu, ah & 0x00f000f0u, bh & 0x00f000f0u, qb[2 * j + 1][0],
                     qb[2 * j + 1][1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t base = kst + (2 * pair + i) * kQ4TileBytes + par_off;
          const float2 sz0 = h2_to_f2(lds32(base)), sz1 = h2_to_f2(lds32(base + 8 * kQ4ParamBytes));
          float x[4];  // s_g acc_g of [half][head]
          f32x2_unpack(f32x2_mul(f32x2_pack(c[i][0], c[i][1]), f32x2_pack(sz0.x * kc[0], sz0.x * kc[1])), x[0], x[1]);
          f32x2_unpack(f32x2_mul(f32x2_pack(c[i][2], c[i][3]), f32x2_pack(sz1.x * kc[0], sz1.x * kc[1])), x[2], x[3]);
#pragma unroll
          for (int h = 0; h < G; ++h) {
            // the sum over the groups (the four lanes t) as a product with ones, plus z . sum q
            float d[4];
            const uint32_t h0 = __float_as_uint(x[h]) & kTf32Mask, h1 = __float_as_uint(x[2 + h]) & kTf32Mask;
            mma1688_tf32_from(d, __float_as_uint(sz0.y), __float_as_uint(sz1.y), __float_as_uint(sz0.y),
                              __float_as_uint(sz1.y), qs_b[h][0], qs_b[h][1], from[h]);
            mma1688_tf32(d, h0, h1, __float_as_uint(x[h] - __uint_as_float(h0)),
                         __float_as_uint(x[2 + h] - __uint_as_float(h1)), kOne, kOne);
            lg[h][2 * pair + i][0] = d[0];
            lg[h][2 * pair + i][1] = d[2];
          }
        }
      }
      __syncwarp();  // every lane has read K and its flags
      issue_k();
      if (!__all_sync(0xffffffffu, mbar_try_wait(v_full, done & 1)) && !wait_warp(v_full, done & 1, p.err)) break;
      if (flags & kNew) {
        const int lane16 = lane & 15, j = lane16 >> 2, tt = lane16 & 3, tok = (ntok - 1) % kQ4Tile;
        const uint32_t tile = v_buf + (ntok - 1) / kQ4Tile * kQ4TileBytes;
        if (lane >= 16) {
          sts32(tile + q4_v_word(tok, j, tt), new_codes);
          if (tt == 0) sts32(tile + q4_param(tok, j), new_par);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }

      if (ntok > 0) {
        // V's scale and minimum of this lane's tokens and group
        uint32_t vp[kUnitTiles][2];
#pragma unroll
        for (int tile = 0; tile < kUnitTiles; ++tile)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            vp[tile][half] = lds32(v_buf + tile * kQ4TileBytes + par_off + half * 8 * kQ4ParamBytes);
        if (ntok < kUnit) {
          // past the end: no weight, and 0 for whatever the bytes there hold
#pragma unroll
          for (int tile = 0; tile < kUnitTiles; ++tile)
#pragma unroll
            for (int half = 0; half < 2; ++half)
              if (tile * kQ4Tile + 8 * half + r >= ntok) {
                vp[tile][half] = 0u;
#pragma unroll
                for (int h = 0; h < G; ++h) lg[h][tile][half] = -INFINITY;
              }
        }
        // ---- running maximum: moves only when a logit passes it by more than 8 (2^8 of headroom) ----
        float top[G];
        bool moved = false;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          top[h] = fmaxf(lg[h][0][0], lg[h][0][1]);
#pragma unroll
          for (int tile = 1; tile < kUnitTiles; ++tile) top[h] = fmax3(top[h], lg[h][tile][0], lg[h][tile][1]);
          moved |= top[h] > 8.f || m[h] == -INFINITY;
        }
        moved = __any_sync(0xffffffffu, moved);
        if (moved) {
#pragma unroll
          for (int h = 0; h < G; ++h) {
            float x = top[h];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            // logits are relative to the old maximum (to 0 if there is none yet)
            const bool none = m[h] == -INFINITY;
            const float up = none ? (x == -INFINITY ? 0.f : x) : fmaxf(x, 0.f);
            const float sc = none ? 0.f : ex2_approx(-up);
            m[h] = none ? x : m[h] + up;
            from[h][0] = from[h][1] = from[h][2] = from[h][3] = m[h] == -INFINITY ? 0.f : -m[h];
#pragma unroll
            for (int tile = 0; tile < kUnitTiles; ++tile)
#pragma unroll
              for (int half = 0; half < 2; ++half) lg[h][tile][half] -= up;
            l2[h] = f32x2_mul(l2[h], f32x2_pack(sc, sc));
            z2[h] = f32x2_mul(z2[h], f32x2_pack(sc, sc));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[i][h] *= sc;
              acc[i][2 + h] *= sc;
            }
            if (kCentred) ones[h] *= sc;
          }
        }
        // ---- p and its sums ----
        float2 vsz[kUnitTiles][2];
        float smax = 0.f;
#pragma unroll
        for (int tile = 0; tile < kUnitTiles; ++tile) {
          vsz[tile][0] = h2_to_f2(vp[tile][0]);
          vsz[tile][1] = h2_to_f2(vp[tile][1]);
          smax = fmax3(smax, vsz[tile][0].x, vsz[tile][1].x);
        }
        uint64_t pr[G][kUnitTiles], mid[kUnitTiles];  // mid: z, or the value of the codes' middle
#pragma unroll
        for (int tile = 0; tile < kUnitTiles; ++tile) {
          mid[tile] = f32x2_pack(vsz[tile][0].y, vsz[tile][1].y);
          if (kCentred)
            mid[tile] = f32x2_fma(f32x2_pack(vsz[tile][0].x, vsz[tile][1].x), f32x2_pack(7.5f, 7.5f), mid[tile]);
        }
#pragma unroll
        for (int h = 0; h < G; ++h)
#pragma unroll
          for (int tile = 0; tile < kUnitTiles; ++tile) {
            pr[h][tile] = f32x2_pack(ex2_approx(lg[h][tile][0]), ex2_approx(lg[h][tile][1]));
            l2[h] = f32x2_add(l2[h], pr[h][tile]);
            z2[h] = f32x2_fma(pr[h][tile], mid[tile], z2[h]);
          }
        if (moved || __any_sync(0xffffffffu, smax * nu > 64.f)) {
          // p <= 2^8, so p s nu stays below 2^14 otherwise. nu: the power of two
          // that takes the largest p s of this unit to [1, 2)
          float wmax = 0.f;
#pragma unroll
          for (int h = 0; h < G; ++h)
#pragma unroll
            for (int tile = 0; tile < kUnitTiles; ++tile) {
              float p0, p1;
              f32x2_unpack(pr[h][tile], p0, p1);
              wmax = fmax3(wmax, p0 * vsz[tile][0].x, p1 * vsz[tile][1].x);
            }
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, off));
          const float nu2 = pow2(max(-24, min(24, -exponent_of(wmax))));
          const float sc = __fdividef(nu2, nu);
          nu = nu2;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] *= sc;
          if (kCentred) {
#pragma unroll
            for (int h = 0; h < G; ++h) ones[h] *= sc;
          }
        }
        // ---- o += (p s) . V codes ----
#pragma unroll
        for (int tile = 0; tile < kUnitTiles; ++tile) {
          if (tile == 2 && ntok <= kHalfUnit) break;
          const uint64_t s2 = f32x2_pack(vsz[tile][0].x * nu, vsz[tile][1].x * nu);
          float a0, a1, b0 = 0.f, b1 = 0.f;
          f32x2_unpack(f32x2_mul(pr[0][tile], s2), a0, a1);
          if (G > 1) f32x2_unpack(f32x2_mul(pr[G - 1][tile], s2), b0, b1);
          const uint32_t p0 = movmatrix(pack_f16(a0, b0)), p1 = movmatrix(pack_f16(a1, b1));
          const uint32_t base = v_buf + tile * kQ4TileBytes + v_off;
          if (kCentred) mma16816(ones, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, p0, p1);
          uint32_t lo[4], hi[4];
          ldmatrix_x4_trans(base, lo);
          ldmatrix_x4_trans(base + 8 * kQ4CodeBytes, hi);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t lo8 = lo[q] >> 8, hi8 = hi[q] >> 8;
            mma16816(acc[2 * q], lo[q] & 0x000f000fu, lo[q] & 0x00f000f0u, hi[q] & 0x000f000fu, hi[q] & 0x00f000f0u, p0,
                     p1);
            mma16816(acc[2 * q + 1], lo8 & 0x000f000fu, lo8 & 0x00f000f0u, hi8 & 0x000f000fu, hi8 & 0x00f000f0u, p0, p1);
          }
        }
      }
      ++done;
      __syncwarp();  // every lane has read V
      issue_v(done);
    }

    // ---- the ticket of the item before: its writes have had a unit's time to land ----
    if (pending) {
      pending = false;
      const int first_chunk = sF[pend_b] + pend_b, nch = pend_c >> 16, c = pend_c & 0xffff;
      auto arrive = [&](int64_t ticket, int expected) -> bool {
        __syncwarp();
        int is_last = 0;
        if (lane == 0) {
          __threadfence();
          is_last = atomicAdd(p.tickets + ticket, 1) == expected - 1;
          if (is_last) p.tickets[ticket] = 0;  // ready for the next call
        }
        is_last = __shfl_sync(0xffffffffu, is_last, 0);
        if (is_last) __threadfence();
        return is_last != 0;
      };
      const int g0 = c - c % kFan;  // this chunk's group of kFan
      const int64_t slot_g = static_cast<int64_t>(first_chunk + g0) * p.rows + pend_head;
      const int in_group = min(kFan, nch - g0);
      bool merge = arrive(slot_g, in_group);
      int64_t at = slot_g, stride = p.rows;
      int n = in_group;
      if (merge && nch > kFan) {
        // merge the group into its first slot, then the groups
        float M[G], den[G];
        float4 a[G];
        merge_slots<G>(p, slot_g, p.rows, in_group, lane, M, den, a);
        __syncwarp();  // every lane has read the slot that is overwritten
#pragma unroll
        for (int h = 0; h < G; ++h) {
          reinterpret_cast<float4*>(p.opart + (slot_g * G + h) * kHeadDim)[lane] = a[h];
          if (lane == 0) p.ml[slot_g * G + h] = make_float2(M[h], den[h]);
        }
        at = static_cast<int64_t>(first_chunk) * p.rows + pend_head;
        stride = static_cast<int64_t>(kFan) * p.rows;
        n = (nch + kFan - 1) / kFan;
        merge = arrive(at + p.rows, n);  // the ticket of chunk 1, which no group uses
      }
      if (merge) {
        uint16_t* orow = p.out + (static_cast<int64_t>(pend_b) * p.rows + pend_head) * G * kHeadDim;
        float M[G], den[G];
        float4 a[G];
        merge_slots<G>(p, at, stride, n, lane, M, den, a);
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float inv = den[h] == 0.f ? 0.f : 1.f / den[h];
          uint2 v;
          v.x = Ops::pack(a[h].x * inv, a[h].y * inv);
          v.y = Ops::pack(a[h].z * inv, a[h].w * inv);
          reinterpret_cast<uint2*>(orow + h * kHeadDim)[lane] = v;
        }
      }
    }
    if (!have) break;
    if (!(flags & kLast)) continue;

    // ---- the item's end: lanes with t == (r & 3) hold dims 32 t + 8 q + 4 (r >> 2) .. + 3, q = 0..3 ----
    const int4 it = info->item[items_done & 3];
    ++items_done;
    const int b = it.x, head = it.y, nch = it.z >> 16;
    const int64_t slot = static_cast<int64_t>(sF[b] + b + (it.z & 0xffff)) * p.rows + head;
    const float back = __fdividef(16777216.f, nu);
    const int d0 = 32 * t + 4 * (r >> 2);
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float s0, s1, z0, z1;
      f32x2_unpack(l2[h], s0, s1);
      f32x2_unpack(z2[h], z0, z1);
      float sum = s0 + s1, z = z0 + z1;
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
        z += __shfl_xor_sync(0xffffffffu, z, off);
      }
      if (kCentred) z = fmaf(ones[h], -7.5f / nu, z);
      const float inv = nch > 1 ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
      const float ka = back * inv, kb = ka * 0.0625f;
      z *= inv;
      if (t == (r & 3)) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float o0 = fmaf(acc[2 * q][h], ka, z), o1 = fmaf(acc[2 * q][2 + h], kb, z);
          const float o2 = fmaf(acc[2 * q + 1][h], ka, z), o3 = fmaf(acc[2 * q + 1][2 + h], kb, z);
          if (nch > 1) {
            *reinterpret_cast<float4*>(p.opart + (slot * G + h) * kHeadDim + d0 + 8 * q) = make_float4(o0, o1, o2, o3);
          } else {
            uint16_t* orow = p.out + ((static_cast<int64_t>(b) * p.rows + head) * G + h) * kHeadDim;
            uint2 v;
            v.x = Ops::pack(o0, o1);
            v.y = Ops::pack(o2, o3);
            *reinterpret_cast<uint2*>(orow + d0 + 8 * q) = v;
          }
        }
      }
      if (nch > 1 && lane == 0) p.ml[slot * G + h] = make_float2(m[h], sum);
    }
    pending = nch > 1;
    pend_b = b;
    pend_head = head;
    pend_c = it.z;
  }
  // Only after a wait that ran out: never leave a copy in flight into this CTA's shared
  // memory. Tickets that this warp should have taken are missing, so a later call would
  // merge too early: the workspace is marked, and calls refuse it until it is zero-filled.
  if (done < issued) {
    if (lane == 0) atomicOr(p.work + 1, kSpoilt);
    mbar_wait(v_full, done & 1, p.err);
    for (; done < issued; ++done) mbar_wait(k_full + 8 * (done & 1), (done >> 1) & 1, p.err);
  }

  if (dynamic && lane == 0) {
    // the last warp to take no more items resets the counters for the next call
    __threadfence();
    if (atomicAdd(p.work + 1, 1) == W - 1) {
      p.work[0] = 0;
      p.work[1] = 0;
    }
  }
}

template <int G>
constexpr size_t smem_bytes() {
  return static_cast<size_t>(kWarps) *
             (3 * kUnitBytes + 2 * G * kHeadDim * 2 + sizeof(WarpInfo)) +
         (3 * kMaxSeqs + 1 + (kClasses + 1) * 32) * sizeof(int);
}
static_assert(smem_bytes<2>() <= 227 * 1024, "shared memory above the 227 KB a CTA can opt into");

template <Elem E, int G>
cudaError_t launch_typed(const Q4DecodeParams& p, cudaStream_t stream) {
  static std::atomic<int> sm_count[64];  // 0: this device's attributes are not set yet
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64) sms = sm_count[dev].load(std::memory_order_acquire);
  if (sms == 0) {
    const cudaError_t e = cudaFuncSetAttribute(q4_decode_kernel<E, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem_bytes<G>()));
    if (e != cudaSuccess) return e;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) sms = 152;
    if (dev >= 0 && dev < 64) sm_count[dev].store(sms, std::memory_order_release);
  }
  q4_decode_kernel<E, G><<<sms, kWarps * 32, smem_bytes<G>(), stream>>>(p);
  return cudaGetLastError();
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Most slots for partial results that a launch over these sizes can use: its
// whole chunks, one short chunk per sequence, times heads. chunk_tokens makes at
// most one whole chunk per warp up to x = kMaxChunk, chunks of 17 units or more
// up to x = 256 and of 29 or more beyond; and none shorter than half a unit.
int64_t max_slots(int64_t num_seqs, int64_t rows, int64_t max_ctx) {
  const int64_t units = num_seqs * ((max_ctx + kUnit - 1) / kUnit) * rows;
  const int64_t halves = num_seqs * (max_ctx / kHalfUnit) * rows;
  int64_t chunks = int64_t{256} * 152 * kWarps / 17 + 1;
  if (units / 29 + 1 > chunks) chunks = units / 29 + 1;
  return (halves < chunks ? halves : chunks) + num_seqs * rows;
}

}  // namespace

// Workspace: two work counters and a ticket per slot (zero between calls), then
// the slots' partial outputs and (m, l). Launches of kMaxSeqs sequences follow
// one another on the stream and share it. The counters' region depends on the
// size of the workspace alone, so that calls of other sizes on the same
// workspace find zeros there: 1/128 of it, which holds the tickets (4 bytes) of
// any number of items (520 bytes or more) that fit in the rest.
size_t decode_q4_counter_bytes(size_t workspace_bytes) { return 256 + (workspace_bytes / 128 & ~size_t{255}); }

size_t decode_q4_workspace_bytes(int32_t num_seqs, int32_t hkv, int32_t group, int32_t max_ctx) {
  const int heads = group > 1 ? 2 : 1;  // per item
  const int64_t n = max_slots(num_seqs < kMaxSeqs ? num_seqs : kMaxSeqs, hkv * group / heads, max_ctx);
  const size_t partials = static_cast<size_t>(n) * heads * (kHeadDim * sizeof(float) + sizeof(float2));
  return align_up((partials + 512) / 127 * 128 + 512, 256);
}

cudaError_t launch_decode_q4(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                             int32_t num_blocks, const int32_t* block_tables, int32_t bt_stride,
                             const int32_t* context_lens, int32_t num_seqs, int32_t hkv, int32_t group,
                             int32_t max_ctx, float scale, void* out, void* workspace, size_t workspace_bytes,
                             unsigned int* err, cudaStream_t stream, const FusedStore* fused, Elem elem) {
  for (int32_t b0 = 0; b0 < num_seqs; b0 += kMaxSeqs) {
    Q4DecodeParams p{};
    p.num_seqs = num_seqs - b0 < kMaxSeqs ? num_seqs - b0 : kMaxSeqs;
    p.q = static_cast<const uint16_t*>(q) + b0 * q_row_stride;
    p.q_row_stride = q_row_stride;
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.num_blocks = num_blocks;
    p.hkv = hkv;
    p.block_tables = block_tables + static_cast<int64_t>(b0) * bt_stride;
    p.bt_stride = bt_stride;
    p.context_lens = context_lens + b0;
    p.max_ctx = max_ctx;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = static_cast<uint16_t*>(out) + static_cast<int64_t>(b0) * hkv * group * kHeadDim;
    const int heads = group > 1 ? 2 : 1;
    p.rows = hkv * group / heads;
    p.share = group / heads;
    const int64_t n = max_slots(num_seqs < kMaxSeqs ? num_seqs : kMaxSeqs, p.rows, max_ctx);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.work = reinterpret_cast<int32_t*>(ws);
    p.tickets = p.work + 2;
    ws += decode_q4_counter_bytes(workspace_bytes);
    p.opart = reinterpret_cast<float*>(ws);
    p.ml = reinterpret_cast<float2*>(ws + static_cast<size_t>(n) * heads * kHeadDim * sizeof(float));
    p.max_slots = n;
    if (fused) {
      p.k_new = static_cast<const uint16_t*>(fused->k) + b0 * fused->k_row_stride;
      p.v_new = static_cast<const uint16_t*>(fused->v) + b0 * fused->v_row_stride;
      p.k_new_stride = fused->k_row_stride;
      p.v_new_stride = fused->v_row_stride;
      p.slot_mapping = fused->slot_mapping + b0;
      p.k_cache_w = static_cast<uint8_t*>(const_cast<void*>(k_cache));
      p.v_cache_w = static_cast<uint8_t*>(const_cast<void*>(v_cache));
    }
    p.err = err;
    const bool f16 = elem == Elem::kF16;
    const cudaError_t e = heads == 1 ? (f16 ? launch_typed<Elem::kF16, 1>(p, stream) : launch_typed<Elem::kBF16, 1>(p, stream))
                                     : (f16 ? launch_typed<Elem::kF16, 2>(p, stream) : launch_typed<Elem::kBF16, 2>(p, stream));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pkv
