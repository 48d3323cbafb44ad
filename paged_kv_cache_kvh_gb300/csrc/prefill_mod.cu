// prefill_mod.cu -- variable-length prefill attention whose scores are capped or biased by distance and whose rows each
// see a range of keys, for any head counts, on tcgen05 tensor cores.
//
// Query row i of sequence b sits at position p = Lk_b - Lq_b + i. With x = scale * q.k_t:
//   z_t = [cap * tanh(x / cap) or x] - slope_h * |p - t|
//   out = sum e^(z_t - m) v_t / sum e^(z_t - m)   over lo <= t < hi,
//   lo = max(key_start of the row, p - window + 1, 0),  hi = min(Lk, max(p + 1, prefix of the sequence)).
// Every mask here (causal, window, document, prefix) leaves a row one range of keys, so a CTA goes over the key tiles
// between its rows' smallest lo and largest hi and nothing else; a warp (32 rows) masks single scores only in tiles that
// one of its rows' ranges ends in, and writes zeros without any arithmetic for tiles that none of its rows sees.
//
// The machine is that of the causal kernel without modifications: two softmax groups, 128 query rows each, one issuing
// thread, one TMA warp, a ring of three 32 KB tiles; but eight warps to a group, two threads to a row (four to a group
// left each scheduler too little to hide the waits behind: 5000 capped rows on 7001 403 us instead of 369). The two
// groups are two query heads of one kv head at the same rows, or, where a kv head has an odd number of query heads, one
// head at two neighbouring tiles of rows: either way one K and one V tile serves both.
//
// What bounds it: a key tile of both groups takes about 2 us, its products 1.1 of that; the rest is the chain of each
// group (product, softmax, barrier, product) with two groups to overlap and the softmax's issue slots, 54 % in use as
// the tensor pipe is. 16 on 8 heads, 5000 on 7001 in the cache: 350 us capped at 50 and 311 without a cap, of 207 at
// cuBLAS' rate (0.59 and 0.67 of it); 16 k rows of 100..1024-token prompts with a cap and a window: 77 us, 3.5 us fixed
// per CTA among it. Measured and not kept: 384 threads with registers shared out by role (427 us where 404 was), scores
// fetched a tile ahead (430: three slots of the ring are too few for it), a CTA going from item to item with the next
// one's first products under the last one's end (538: the loop over items around the softmax makes the compiler spill).
//
// tanh: the softmax is issue-limited, and tanh through exponential and reciprocal would triple its special function
// work (128 x 128 scores a group: 2 us a tile of 1.6). An odd polynomial on packed pairs costs 4 instructions a pair for
// bf16 where all of a warp's |x| <= 0.4 cap, 6 up to the cap (fp16: one more each); only a tile with scores beyond goes
// through 1 - 2 / (1 + e^2x). A score is off by at most 7e-6 of itself for bf16 (p by 2^-12 at a score of 32, where its
// rounding to 16 bits loses 2^-9) and 6e-7 for fp16 (2^-15; 2^-12).
//
// The maximum: rows go by a reference that is moved when a score passes it by 2^8 and subtracted where the scores are
// scaled, so a tile needs one pass for the largest value and nothing else. Scores of bf16 rows capped at 52 or less
// need none at all: 2^z lies within 2^-75 .. 2^75, sums of it times v within fp32 (|v| up to 2^52; beyond, the row is
// computed again, see below), and bf16 keeps the same relative precision there as near 1.
//
// Values of V at keys that a row does not see are multiplied by p = 0; where they are not finite the sum is spoilt
// (0 * NaN). The rows of V behind the sequence's end, which may hold anything, are zeroed in shared memory. Elsewhere
// such values are rare, so they are found in the result: a row whose sum is not finite is computed once more by its
// warp from the rows in memory, one key to a lane, with the keys that it does not see left out.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>

#include <cuda.h>

#include "pkv_common.cuh"

namespace pkv {

struct PrefillModArgs {
  const void* q;
  int64_t q_row_stride;
  int32_t total_q;
  const void* k;  // contiguous keys, or the caches where block_tables is given
  const void* v;
  int64_t kv_row_stride;
  int32_t total_k;
  int32_t num_blocks;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int32_t max_seqlen_q, max_seqlen_k;
  const int32_t* block_tables;
  int32_t bt_stride;
  int32_t num_seqs, hq, hkv;
  float scale, softcap;
  const float* slopes;
  int32_t window;
  const int32_t* key_starts;
  const int32_t* prefix_lens;
  void* out;
};

namespace {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kTileBytes = 128 * kHeadDim * 2;  // 32 KB
constexpr int kHalfBytes = kTileBytes / 2;      // 16 KB: 128 rows x 64 dims
constexpr int kKvSlots = 3;
constexpr int kSoftmaxWarps = 16;                // 8 to a group: two threads share a row, 64 of its keys (and dims) each
constexpr int kThreads = (4 + kSoftmaxWarps) * 32;
constexpr int kCols = kBN / 2;                   // scores to a thread
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kOffQ = 0;                                // 2 tiles
constexpr int kOffP = 2 * kTileBytes;                   // 2 tiles
constexpr int kOffKV = 4 * kTileBytes;                  // kKvSlots tiles
constexpr int kOffBar = kOffKV + kKvSlots * kTileBytes;  // barriers
constexpr int kBarQ = 0;
constexpr int kBarKvFull = 1;                     // +slot
constexpr int kBarKvFree = kBarKvFull + kKvSlots;
constexpr int kBarSFull = kBarKvFree + kKvSlots;  // +group
constexpr int kBarPReady = kBarSFull + 2;         // +group
constexpr int kBarOFinal = kBarPReady + 2;
constexpr int kBarVTail = kBarOFinal + 1;
constexpr int kBarDrain = kBarVTail + 1;
constexpr int kBarStaged = kBarDrain + 1;         // the softmax warps have staged their O rows
constexpr int kNumBars = kBarStaged + 1;
constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tmem address, abort flag, smallest lo and largest hi of 32 rows,
constexpr int kMiscBytes = 8 + 16 * 4 + 8 * 4;    // rows to be computed once more
constexpr int kOffMax = kOffMisc + kMiscBytes;    // [group][half][row] bf16: the halves' largest scores
constexpr size_t kSmemBytes = kOffMax + 4 * kBM * 2 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "shared memory above the 227 KB a CTA can opt into");

// tanh x = x (c0 + c1 x^2 + ...), least-maximum fits of tanh(x) / x: for bf16 off by 6.3e-6 of the result for |x| <= 0.4
// and 6.9e-6 for |x| <= 1, for fp16 by 5.6e-7 for |x| <= 0.5 and 6.1e-7 for |x| <= 1.
template <Elem E>
struct TanhFit;
template <>
struct TanhFit<Elem::kBF16> {
  static constexpr int kNear = 3, kFar = 5;
  static constexpr double kNearTop = 0.4, kFarTop = 1.0;
  static constexpr double kNearC[6] = {0.9999937530753578, -0.33262579162588246, 0.12127784712702376};
  static constexpr double kFarC[6] = {0.9999930890836747, -0.3329806490410056, 0.13036809964236198,
                                      -0.04481753658422978, 0.009036415875549408};
};
template <>
struct TanhFit<Elem::kF16> {
  static constexpr int kNear = 4, kFar = 6;
  static constexpr double kNearTop = 0.5, kFarTop = 1.0;
  static constexpr double kNearC[6] = {0.9999994557571216, -0.33326317896947046, 0.13190296288204925,
                                       -0.044402218547957305};
  static constexpr double kFarC[6] = {0.9999994135741078,    -0.3332904232451419,  0.13281433250603616,
                                      -0.051605653809187996, 0.016743090747062123, -0.0030670504021806768};
};
constexpr float kNoCap = 1e30f;     // from here on a cap changes no score that fp32 tells from its neighbours below 1e26
constexpr float kFixedCap = 52.f;  // bf16: scores capped here and below need no running maximum

struct PrefillModParams {
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* block_tables;
  int32_t bt_stride, num_blocks, num_seqs;
  int32_t q_tiles;        // tiles of 128 rows (pairs of them where the groups are neighbours) a sequence has at most
  int32_t max_seqlen_q, max_seqlen_k, total_q, total_k;
  int32_t paged;
  int32_t hq, group;      // query heads; per kv head
  int32_t neighbours;     // the two softmax groups are neighbouring tiles of one head, not two heads
  int32_t units;          // head pairs, or heads
  int32_t first;          // this launch's first item
  float scale, scale_log2;
  float softcap;
  float cap_log2, scale_by_cap;
  float near_top, far_top;      // largest |q.k| that the polynomials take (0: none but zeros)
  float near_c[6], far_c[6];    // of z in log2 units, by powers of q.k
  float tanh_c[6];              // kFarC
  int32_t fixed;                // no running maximum
  const float* slopes;
  int32_t window;
  const int32_t* key_starts;
  const int32_t* prefix_lens;
  const uint16_t* q;      // once more, for rows that are computed again
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, kv_stride;
  uint16_t* out;
  unsigned int* err;
};

// Bounded wait that also gives up as soon as another role of the CTA has
// aborted (so one lost arrival costs one time-out, not one per wait).
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                              unsigned int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      flag_error(err, PKV_DEVERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}

// 8-column TMEM load / store (32 lanes x 8 x 32 bit), for the rare O rescale
// while the tile's 128 probabilities are still held in registers.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// keeps uses of a tmem_ld8 result after the tcgen05.wait::ld that completes it
__device__ __forceinline__ void tmem_reg_fence8(uint32_t (&r)[8]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * tanh(x / cap) in log2 units, for any x = q.k; the polynomial where the difference from 1 would lose bits
template <int N>
__device__ __forceinline__ float capped(float x, const PrefillModParams& p) {
  const float t = x * p.scale_by_cap, v = t * t;
  float r = p.tanh_c[N - 1];
#pragma unroll
  for (int i = N - 2; i >= 0; --i) r = fmaf(r, v, p.tanh_c[i]);
  const float far = fmaf(-2.f, rcp_approx(1.f + ex2_approx(t * (2.f * kLog2e))), 1.f);
  return p.cap_log2 * (fabsf(t) <= 1.f ? t * r : far);
}
template <int N>
struct Poly2 {  // the polynomial of a pair, plus `add`
  uint64_t c[N];
  __device__ __forceinline__ explicit Poly2(const float* coef) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = f32x2_pack(coef[i], coef[i]);
  }
  __device__ __forceinline__ uint64_t operator()(uint64_t x, uint64_t add) const {
    const uint64_t v = f32x2_mul(x, x);
    uint64_t r = c[N - 1];
#pragma unroll
    for (int i = N - 2; i >= 0; --i) r = f32x2_fma(r, v, c[i]);
    return f32x2_fma(x, r, add);
  }
};
__device__ __forceinline__ float max_all(const float (&s)[kCols]) {
  float a = s[0], b = s[1];
#pragma unroll
  for (int j = 2; j < kCols - 2; j += 4) {
    a = fmax3(a, s[j], s[j + 1]);
    b = fmax3(b, s[j + 2], s[j + 3]);
  }
  return fmaxf(fmax3(a, s[kCols - 2], s[kCols - 1]), b);
}
__device__ __forceinline__ float size_all(const float (&s)[kCols]) {  // the largest |s|
  float a = fabsf(s[0]), b = fabsf(s[1]);
#pragma unroll
  for (int j = 2; j < kCols - 2; j += 4) {
    a = fmax3(a, fabsf(s[j]), fabsf(s[j + 1]));
    b = fmax3(b, fabsf(s[j + 2]), fabsf(s[j + 3]));
  }
  return fmaxf(fmax3(a, fabsf(s[kCols - 2]), fabsf(s[kCols - 1])), b);
}

// One (row, query head) by a whole warp from the rows in memory: a key to a lane, then four dims to a lane.
template <Elem E>
__device__ __noinline__ void row_again(const PrefillModParams& p, int b, int64_t k0, int64_t row, int head, int pos,
                                       int lo, int hi, int lane) {
  using Ops = ElemOps<E>;
  const int hk = head / p.group;
  const uint16_t* q = p.q + row * p.q_stride + head * kHeadDim;
  const float slope = p.slopes ? p.slopes[head] * kLog2e : 0.f;
  auto key_row = [&](int t) -> int64_t {
    if (!p.paged) return (k0 + t) * p.kv_stride + hk * kHeadDim;
    int blk = p.block_tables[static_cast<int64_t>(b) * p.bt_stride + t / kBlockSize];
    if (blk < 0 || blk >= p.num_blocks) blk = 0;  // reported where the tile was fetched
    return (static_cast<int64_t>(blk) * kBlockSize + t % kBlockSize) * p.kv_stride + hk * kHeadDim;
  };
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int t0 = lo; t0 < hi; t0 += 32) {
    const int t = t0 + lane;
    float z = -INFINITY;
    if (t < hi) {
      const uint4* kr = reinterpret_cast<const uint4*>(p.k + key_row(t));
      float x = 0.f;
      for (int i = 0; i < kHeadDim / 8; ++i) {
        const uint4 a = kr[i], c = reinterpret_cast<const uint4*>(q)[i];
        x = fmaf(Ops::lo(a.x), Ops::lo(c.x), fmaf(Ops::hi(a.x), Ops::hi(c.x), x));
        x = fmaf(Ops::lo(a.y), Ops::lo(c.y), fmaf(Ops::hi(a.y), Ops::hi(c.y), x));
        x = fmaf(Ops::lo(a.z), Ops::lo(c.z), fmaf(Ops::hi(a.z), Ops::hi(c.z), x));
        x = fmaf(Ops::lo(a.w), Ops::lo(c.w), fmaf(Ops::hi(a.w), Ops::hi(c.w), x));
      }
      z = p.softcap > 0.f ? p.cap_log2 * tanhf(x * p.scale_by_cap) : x * p.scale_log2;
      z = fmaf(-slope, fabsf(static_cast<float>(pos - t)), z);
    }
    float top = fmaxf(m, z);
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float use = top == -INFINITY ? 0.f : top;
    const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - use);
    const float e = t < hi ? ex2_approx(z - use) : 0.f;
    float sum = e;
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    m = top;
    l = l * alpha + sum;
    for (int i = 0; i < 4; ++i) acc[i] *= alpha;
    const int n = min(32, hi - t0);
    for (int i = 0; i < n; ++i) {
      const float pi = __shfl_sync(0xffffffffu, e, i);
      const uint2 x = *(reinterpret_cast<const uint2*>(p.v + key_row(t0 + i)) + lane);
      acc[0] = fmaf(pi, Ops::lo(x.x), acc[0]);
      acc[1] = fmaf(pi, Ops::hi(x.x), acc[1]);
      acc[2] = fmaf(pi, Ops::lo(x.y), acc[2]);
      acc[3] = fmaf(pi, Ops::hi(x.y), acc[3]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *(reinterpret_cast<uint2*>(p.out + (row * p.hq + head) * kHeadDim) + lane) =
      make_uint2(Ops::pack(acc[0] * inv, acc[1] * inv), Ops::pack(acc[2] * inv, acc[3] * inv));
}

// The cluster of CTAs that split the keys of one item (kSplit).
__device__ __forceinline__ int cluster_parts() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_part() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// this CTA's shared address -> the same place in another CTA of the cluster
__device__ __forceinline__ uint32_t in_part(uint32_t addr, int part) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(part));
  return r;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_f4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}

// The launch of split items may begin while the one before it still runs, and must not be over before that is.
__device__ __forceinline__ void wait_for_others() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// kSplit: the CTAs of a cluster have parts of one item's keys.
template <Elem E, bool kCap, bool kBias, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_mod_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PrefillModParams p) {
  using Ops = ElemOps<E>;
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte alignment for the 128-byte-swizzle atoms.
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_addr);
  const uint32_t bar0 = sbase + kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* s_lo = reinterpret_cast<int*>(smem + kOffMisc + 8);               // [8] smallest lo of 32 rows
  int* s_hi = s_lo + 8;                                                  // [8] largest hi
  uint32_t* s_again = reinterpret_cast<uint32_t*>(s_hi + 8);             // [2][4] rows to be computed once more

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // ---- work item: (query tile, sequence, heads), the last query tiles (the longest key ranges) first ----
  if (!kSplit) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // items split over clusters fill the end
  const int parts = kSplit ? cluster_parts() : 1, part = kSplit ? cluster_part() : 0;
  const int item = p.first + static_cast<int>(blockIdx.x) / parts;
  const int per_tile = p.num_seqs * p.units;
  const int qt = p.q_tiles - 1 - item / per_tile;
  const int b = (item % per_tile) / p.units, unit = item % p.units;
  const int head0 = p.neighbours ? unit : 2 * unit;
  const int hk = head0 / p.group;

  const int cq0 = p.cu_q[b], cq1 = p.cu_q[b + 1];
  const int ck0 = p.cu_k[b], ck1 = p.cu_k[b + 1];
  const int Lq = cq1 - cq0, Lk = ck1 - ck0;
  const bool bad = Lq < 0 || Lk < Lq || Lq > p.max_seqlen_q || Lk > p.max_seqlen_k || cq0 < 0 || cq1 > p.total_q ||
                   (p.paged ? Lk > static_cast<int64_t>(p.bt_stride) * kBlockSize : (ck0 < 0 || ck1 > p.total_k));
  if (bad) {
    if (threadIdx.x == 0 && qt == 0 && unit == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
    if (kSplit) wait_for_others();
    return;
  }
  const int r0 = qt * (p.neighbours ? 2 * kBM : kBM);
  if (r0 >= Lq) {
    if (kSplit) wait_for_others();
    return;
  }

  // The softmax thread of a row: its position and the keys it sees. Rows behind the last one take its place.
  const int g = (warp - 4) >> 3, half = (warp >> 2) & 1 ? 0 : 1;  // warps 4..7 and 12..15 take the first keys of a tile
  const int rows32 = 4 * g + (warp & 3);                           // the warp's 32 rows, of 8 times 32
  const int row = (warp & 3) * 32 + lane;  // within the group's tile == TMEM lane
  const int g_row0 = r0 + (p.neighbours && g > 0 ? kBM : 0);
  auto seen_from = [&](int r, int& pos_, int& lo_, int& hi_) {  // r: row of the sequence
    r = min(r, Lq - 1);
    pos_ = Lk - Lq + r;
    lo_ = p.window > 0 ? max(0, pos_ - p.window + 1) : 0;
    if (p.key_starts) lo_ = max(lo_, p.key_starts[cq0 + r]);
    hi_ = min(Lk, max(pos_ + 1, p.prefix_lens ? p.prefix_lens[b] : 0));
  };
  int pos = 0, lo = 0, hi = 0, any_lo = 0, any_hi = 0;  // seen by the row; by any of the warp's rows
  if (warp >= 4) {
    seen_from(g_row0 + row, pos, lo, hi);
    // a row without keys widens nothing
    any_lo = __reduce_min_sync(0xffffffffu, lo < hi ? lo : INT32_MAX);
    any_hi = __reduce_max_sync(0xffffffffu, lo < hi ? hi : 0);
    if (lane == 0 && half == 0) {
      s_lo[rows32] = any_lo;
      s_hi[rows32] = any_hi;
      s_again[rows32] = 0;
    }
  }

  // ---- the key tiles ----
  int tile0 = 0, n_tiles = 0;  // a split item's part may have none
  auto set_tiles = [&](int first_key, int end_key) {
    // rows that see nothing at all: one tile, all masked
    const int all_tiles = first_key < end_key ? (end_key + kBN - 1) / kBN - first_key / kBN : 1;
    tile0 = (first_key < end_key ? first_key / kBN : 0) + (kSplit ? all_tiles * part / parts : 0);
    n_tiles = kSplit ? all_tiles * (part + 1) / parts - all_tiles * part / parts : all_tiles;
  };
  // Tile n of this CTA's. A bias favours the nearest keys: from the last tile to the first, the reference is found in the
  // first one and stays (5000 on 7001: 404 us from the first on, 331 from the last; without a bias 308 and 326).
  constexpr bool kBack = kBias;
  auto first_key_of = [&](int n) { return (tile0 + (kBack ? n_tiles - 1 - n : n)) * kBN; };
  auto k_row = [&](int n) -> int {  // where tile n begins
    const int key0 = first_key_of(n);
    if (!p.paged) return ck0 + key0;
    int blk = p.block_tables[static_cast<int64_t>(b) * p.bt_stride + key0 / kBlockSize];
    if (blk < 0 || blk >= p.num_blocks) {
      flag_error(p.err, PKV_DEVERR_BAD_BLOCK);
      blk = 0;
    }
    return blk * kBlockSize + key0 % kBlockSize;
  };
  // ring item i: K of tile i / 2 (even i) or V (odd i), into slot i % kKvSlots
  auto load_kv = [&](int i) {
    const int slot = i % kKvSlots;
    const CUtensorMap* tm = (i & 1) ? &tm_v : &tm_k;
    const int at = k_row(i >> 1);
    const uint32_t dst = sbase + kOffKV + slot * kTileBytes;
    mbar_arrive_expect_tx(bar(kBarKvFull + slot), kTileBytes);
    tma_load_3d(dst, tm, 0, hk, at, bar(kBarKvFull + slot));
    tma_load_3d(dst + kHalfBytes, tm, 64, hk, at, bar(kBarKvFull + slot));
  };
  // Without first keys of single rows every row sees at least itself, and the range follows from the first and last row.
  if (!p.key_starts) {
    const int pos0 = Lk - Lq + r0, last = Lk - Lq + min(r0 + (p.neighbours ? 2 * kBM : kBM), Lq);
    set_tiles(p.window > 0 ? max(0, pos0 - p.window + 1) : 0, min(Lk, max(last, p.prefix_lens ? p.prefix_lens[b] : 0)));
  }

  // Thread 0 is the TMA warp's issuing lane: the queries and, where their place is known, the first keys and values are on
  // their way before anything else is set up.
  int issued = 0;  // ring items (thread 0)
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bar(i), i == kBarStaged ? kSoftmaxWarps : (i == kBarPReady || i == kBarPReady + 1 ? 8 : 1));
    *s_abort = 0;
    mbar_fence_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    mbar_arrive_expect_tx(bar(kBarQ), 2 * kTileBytes);
    for (int i = 0; i < 2; ++i) {
      const uint32_t dst = sbase + kOffQ + i * kTileBytes;
      const int head = head0 + (p.neighbours ? 0 : i), first = cq0 + r0 + (p.neighbours ? i * kBM : 0);
      tma_load_3d(dst, &tm_q, 0, head, first, bar(kBarQ));
      tma_load_3d(dst + kHalfBytes, &tm_q, 64, head, first, bar(kBarQ));
    }
    for (; issued < kKvSlots && issued < 2 * n_tiles; ++issued) load_kv(issued);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncwarp();  // warp 0 arrives converged, after thread 0 has initialised the barriers
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (p.key_starts) {
    int first_key = INT32_MAX, end_key = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      first_key = min(first_key, s_lo[i]);
      end_key = max(end_key, s_hi[i]);
    }
    set_tiles(first_key, end_key);
  }
  const int tail_keys = Lk - (tile0 + n_tiles - 1) * kBN;  // keys that the last tile has
  const bool v_tail = tail_keys < kBN && n_tiles > 0;
  const int tail_item = kBack ? 1 : 2 * n_tiles - 1;       // the ring item of its values

  if (warp == 0) {
    // =========================== TMA producer ===========================
    auto issue_up_to = [&](int end) {
      if (lane == 0) {
        for (int i = issued; i < end; ++i) {
          const int slot = i % kKvSlots;
          if (i >= kKvSlots && !wait_or_abort(bar(kBarKvFree + slot), ((i / kKvSlots) - 1) & 1, s_abort, p.err))
            break;
          load_kv(i);
          ++issued;
        }
      }
      issued = __shfl_sync(0xffffffffu, issued, 0);
    };
    issue_up_to(kBack ? min(kKvSlots, 2 * n_tiles) : 2 * n_tiles);
    if (v_tail && issued > tail_item) {
      // Zero the rows of the sequence's last V tile that lie past its end.
      const int slot = tail_item % kKvSlots;
      const bool ok = wait_or_abort(bar(kBarKvFull + slot), (tail_item / kKvSlots) & 1, s_abort, p.err);
      if (ok) {
        const uint32_t base = sbase + kOffKV + slot * kTileBytes;
        // rows tail_keys..127 of both 64-dim halves: 128-byte rows, swizzle
        // only permutes 16-byte chunks within a row.
        const int nz = (kBN - tail_keys) * 2 * 8;  // 16-byte chunks
        for (int c = lane; c < nz; c += 32) {
          const int at = tail_keys + (c >> 4);
          const int half_ = (c >> 3) & 1;
          const int chunk = c & 7;
          sts128(base + half_ * kHalfBytes + at * 128 + chunk * 16, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarVTail));
    }
    issue_up_to(2 * n_tiles);
    if (lane == 0) {
      // Never leave a copy in flight into this CTA's shared memory.
      mbar_wait(bar(kBarQ), 0, p.err);
      for (int i = max(0, issued - kKvSlots); i < issued; ++i)
        mbar_wait(bar(kBarKvFull + i % kKvSlots), (i / kKvSlots) & 1, p.err);
    }
  } else if (warp == 1) {
    // =========================== MMA issuer ===========================
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_f16kind_f32(kBM, kBN, false, false, Ops::kMmaFormat);
      constexpr uint32_t idesc_pv = idesc_f16kind_f32(kBM, kHeadDim, false, true, Ops::kMmaFormat);
      bool ok = wait_or_abort(bar(kBarQ), 0, s_abort, p.err);
      auto slot_of = [](int i) { return i % kKvSlots; };
      auto par_of = [](int i) { return static_cast<uint32_t>((i / kKvSlots) & 1); };
      // Descriptor low halves: each product below costs two 32-bit adds and
      // the tcgen05.mma (this one thread issues every product of the CTA).
      const uint32_t lo_kmaj = desc_lo(sbase, 16), lo_v = desc_lo(sbase, kHalfBytes);
      auto issue_s = [&](int i, int n) {
        const uint32_t qa = lo_kmaj + ((kOffQ + i * kTileBytes) >> 4);
        const uint32_t kbb = lo_kmaj + (kOffKV >> 4) + slot_of(2 * n) * (kTileBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < kHeadDim / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
          mma_f16kind_lo(tmem + i * 128, qa + off, kbb + off, idesc_s, ks > 0 ? 1u : 0u);
        }
      };
      auto issue_pv = [&](int i, int n) {
        const uint32_t pa = lo_kmaj + ((kOffP + i * kTileBytes) >> 4);
        const uint32_t vbb = lo_v + (kOffKV >> 4) + slot_of(2 * n + 1) * (kTileBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < kBN / 16; ++ks) {
          const uint32_t aoff = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
          mma_f16kind_lo(tmem + 256 + i * 128, pa + aoff, vbb + ((ks * 16 * 128) >> 4), idesc_pv,
                         (n > 0 || ks > 0) ? 1u : 0u);
        }
      };
      const bool any = !kSplit || n_tiles > 0;
      if (ok && any) ok = wait_or_abort(bar(kBarKvFull + slot_of(0)), par_of(0), s_abort, p.err);
      if (ok && any) {
        tc_fence_after();
        issue_s(0, 0);
        mma_commit(bar(kBarSFull + 0));
        issue_s(1, 0);
        mma_commit(bar(kBarSFull + 1));
        mma_commit(bar(kBarKvFree + slot_of(0)));
      }
      for (int n = 0; ok && n < n_tiles; ++n) {
        const int iv = 2 * n + 1;
        if (iv == tail_item && v_tail)
          ok = wait_or_abort(bar(kBarVTail), 0, s_abort, p.err);
        else
          ok = wait_or_abort(bar(kBarKvFull + slot_of(iv)), par_of(iv), s_abort, p.err);
        if (!ok) break;
        if (!(ok = wait_or_abort(bar(kBarPReady + 0), n & 1, s_abort, p.err))) break;
        tc_fence_after();
        issue_pv(0, n);
        const bool more = n + 1 < n_tiles;
        if (more) {
          if (!(ok = wait_or_abort(bar(kBarKvFull + slot_of(2 * n + 2)), par_of(2 * n + 2), s_abort, p.err)))
            break;
          tc_fence_after();
          issue_s(0, n + 1);
          mma_commit(bar(kBarSFull + 0));
        }
        if (!(ok = wait_or_abort(bar(kBarPReady + 1), n & 1, s_abort, p.err))) break;
        tc_fence_after();
        issue_pv(1, n);
        mma_commit(bar(kBarKvFree + slot_of(iv)));
        if (more) {
          issue_s(1, n + 1);
          mma_commit(bar(kBarSFull + 1));
          mma_commit(bar(kBarKvFree + slot_of(2 * n + 2)));
        }
      }
      mma_commit(bar(kBarOFinal));
      if (!ok) {
        // make sure no product is still writing TMEM before it is released
        mma_commit(bar(kBarDrain));
        mbar_wait(bar(kBarDrain), 0, p.err);
      }
    }
  } else if (warp >= 4) {
    // =========================== softmax groups ===========================
    const int head = head0 + (p.neighbours ? 0 : g);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + g * 128 + half * kCols;
    const uint32_t tO = tmem + lane_base + 256 + g * 128 + half * kCols;
    const uint32_t prow = sbase + kOffP + g * kTileBytes + half * kHalfBytes + row * 128;
    const int swz = row & 7;
    const float sl2 = p.scale_log2;
    const float slope = kBias ? p.slopes[head] * kLog2e : 0.f;
    const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);  // seen by all rows
    const int min_pos = __reduce_min_sync(0xffffffffu, pos);
    __nv_bfloat16* s_max = reinterpret_cast<__nv_bfloat16*>(smem + kOffMax) + 2 * g * kBM + row;  // [half][row]
    // Named barrier of the two warps. Both come to it once per tile and once at the end, whatever happens, so it needs no
    // time limit.
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + rows32) : "memory"); };
    const bool by_maximum = !kCap || kBias || !p.fixed;
    float m = -INFINITY;  // the row's reference, log2 units; within 8 of its running maximum from below, or fixed at 0
    float l = 0.f;        // of this thread's keys
    bool ok = true;
    for (int n = 0; n < n_tiles; ++n) {
      // every lane waits (each needs the acquire); the warp then agrees, so
      // the warp-collective tensor-memory loads below run on all 32 lanes
      if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(bar(kBarSFull + g), n & 1, s_abort, p.err));
      if (!ok) {  // the other warp of these rows may still come to the pair's barrier
        if (by_maximum) pair_sync();
        continue;
      }
      tc_fence_after();
      const int key0 = first_key_of(n) + half * kCols;
      const bool none = key0 + kCols <= any_lo || key0 >= any_hi;  // no row sees any of these keys
      float s[kCols], mx = -INFINITY;
      const float base = m == -INFINITY ? 0.f : m;
      if (!none) {
        {
          uint32_t x0[32], x1[32];
          tmem_ld32(tS + 0, x0);
          tmem_ld32(tS + 32, x1);
          tmem_wait_ld();
          tmem_reg_fence(x0);
          tmem_reg_fence(x1);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            s[j] = __uint_as_float(x0[j]);
            s[32 + j] = __uint_as_float(x1[j]);
          }
        }
        auto each = [&](auto arg) {
#pragma unroll
          for (int j = 0; j < kCols; j += 2) f32x2_unpack(arg(j, f32x2_pack(s[j], s[j + 1])), s[j], s[j + 1]);
        };
        // ---- s = z - base, base the row's reference so far (0 as long as it has seen no key) ----
        const uint64_t neg = f32x2_pack(-base, -base);
        if (kCap) {
          using Fit = TanhFit<E>;
          if (key0 + kCols > Lk) {  // whatever lies behind the sequence has no say in how its scores are worked out
#pragma unroll
            for (int j = 0; j < kCols; ++j) s[j] = j < Lk - key0 ? s[j] : 0.f;
          }
          const float size = size_all(s);
          if (__all_sync(0xffffffffu, size <= p.near_top)) {
            const Poly2<Fit::kNear> poly(p.near_c);
            each([&](int, uint64_t x) { return poly(x, neg); });
          } else if (__all_sync(0xffffffffu, size <= p.far_top)) {
            const Poly2<Fit::kFar> poly(p.far_c);
            each([&](int, uint64_t x) { return poly(x, neg); });
          } else {
#pragma unroll
            for (int j = 0; j < kCols; ++j) s[j] = capped<Fit::kFar>(s[j], p) - base;
          }
        }
        if (kBias) {
          const float less = kCap ? 0.f : base;
          if (key0 + kCols - 1 <= min_pos) {  // all keys at or before all rows: - slope (pos - t) grows by slope a key
            const float first = -slope * static_cast<float>(pos - key0) - less;
            const uint64_t sl2x2 = f32x2_pack(sl2, sl2), step = f32x2_pack(8.f * slope, 8.f * slope);
            uint64_t at[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) at[a] = f32x2_pack(fmaf(slope, 2.f * a, first), fmaf(slope, 2.f * a + 1.f, first));
            each([&](int j, uint64_t x) {
              uint64_t& t = at[(j >> 1) & 3];
              const uint64_t y = kCap ? f32x2_add(x, t) : f32x2_fma(x, sl2x2, t);
              t = f32x2_add(t, step);
              return y;
            });
          } else {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              s[j] = fmaf(-slope, fabsf(static_cast<float>(pos - key0 - j)), kCap ? s[j] : fmaf(s[j], sl2, -less));
          }
        }
        if (!kCap && !kBias) {
          const uint64_t sl2x2 = f32x2_pack(sl2, sl2);
          each([&](int, uint64_t x) { return f32x2_fma(x, sl2x2, neg); });
        }
        if (key0 < all_lo || key0 + kCols > all_hi) {  // some row does not see all of the keys
          const int jlo = lo - key0, jhi = hi - key0;  // this one sees keys j with jlo <= j < jhi
#pragma unroll
          for (int w = 0; w < kCols / 32; ++w) {
            const int a = min(max(jlo - 32 * w, 0), 32), z = min(max(jhi - 32 * w, 0), 32);
            const uint32_t seen = a < z ? (0xffffffffu << a) & (0xffffffffu >> (32 - z)) : 0u;
#pragma unroll
            for (int j = 0; j < 32; ++j) s[32 * w + j] = (seen >> j) & 1u ? s[32 * w + j] : -INFINITY;
          }
        }
        if (by_maximum) mx = max_all(s) + base;
      }
      if (by_maximum) {
        // The reference moves to the row's largest score when that is above it by more than 8 (2^8 of headroom), and to
        // the first tile's in which the row sees a key. Its two threads tell one another theirs (rounded: any value near
        // will do); the place is free again, since the tile's scores are only there once both were done with the last.
        const __nv_bfloat16 mine = __float2bfloat16_rn(mx);
        s_max[half * kBM] = mine;
        pair_sync();
        const float to = fmaxf(__bfloat162float(mine), __bfloat162float(s_max[(half ^ 1) * kBM]));
        const bool move = to > (m == -INFINITY ? m : m + 8.f);
        if (__any_sync(0xffffffffu, move)) {
          const float delta = move ? base - to : 0.f;
          const uint64_t less = f32x2_pack(delta, delta);
#pragma unroll
          for (int j = 0; j < kCols; j += 2) f32x2_unpack(f32x2_add(f32x2_pack(s[j], s[j + 1]), less), s[j], s[j + 1]);
          const float alpha = !move ? 1.f : (m == -INFINITY ? 0.f : ex2_approx(m - to));
          if (move) m = to;
          l *= alpha;
          if (n > 0) {  // the running output too (PV of tile n - 1 is complete: S of tile n was issued after it)
#pragma unroll 1
            for (int c = 0; c < kCols / 8; ++c) {
              uint32_t r[8];
              tmem_ld8(tO + c * 8, r);
              tmem_wait_ld();
              tmem_reg_fence8(r);
#pragma unroll
              for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
              tmem_st8(tO + c * 8, r);
            }
            tmem_wait_st();
          }
        }
      }
      // P = 2^s, rounded to the element type, into the swizzled K-major A tile
      if (!none) {
#pragma unroll
        for (int c = 0; c < kCols / 8; ++c) {
#pragma unroll
          for (int j = c * 8; j < c * 8 + 8; ++j) s[j] = ex2_approx(s[j]);
          const float* e = s + c * 8;
          sts128(prow + ((c ^ swz) << 4), Ops::pack(e[0], e[1]), Ops::pack(e[2], e[3]), Ops::pack(e[4], e[5]),
                 Ops::pack(e[6], e[7]));
        }
      } else {
#pragma unroll
        for (int c = 0; c < kCols / 8; ++c) sts128(prow + ((c ^ swz) << 4), 0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarPReady + g));
      // The row sum is not needed for P: add it up after P is handed over. Where rows may see few keys, of the rounded p,
      // which is what V is multiplied by, so that their shares add up to 1 exactly (a row that sees one key gets its
      // value as it is); in sums over many keys the roundings do not add up (everywhere it would cost 5 to 9 %).
      if (!none) {
        if (key0 < all_lo || key0 + kCols > all_hi) {
#pragma unroll
          for (int j = 0; j < kCols; j += 2) {
            const uint32_t w = Ops::pack(s[j], s[j + 1]);
            s[j] = Ops::lo(w);
            s[j + 1] = Ops::hi(w);
          }
        }
        uint64_t acc[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) acc[a] = f32x2_pack(s[2 * a], s[2 * a + 1]);
#pragma unroll
        for (int j = 8; j < kCols; j += 8)
#pragma unroll
          for (int a = 0; a < 4; ++a) acc[a] = f32x2_add(acc[a], f32x2_pack(s[j + 2 * a], s[j + 2 * a + 1]));
        float t0, t1, t2, t3, t4, t5, t6, t7;
        f32x2_unpack(acc[0], t0, t1);
        f32x2_unpack(acc[1], t2, t3);
        f32x2_unpack(acc[2], t4, t5);
        f32x2_unpack(acc[3], t6, t7);
        l += ((t0 + t1) + (t2 + t3)) + ((t4 + t5) + (t6 + t7));
      }
    }
    if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(bar(kBarOFinal), 0, s_abort, p.err));
    // Epilogue. Every product is complete, so the K/V ring and the two P buffers are free: a row's two threads add up
    // their sums through the one, each stages its half of the normalised O row in the other (the rows of the two groups
    // side by side, 512 B, 16-byte chunks rotated by the row to spread the banks), then each warp stores whole rows.
    const uint32_t stage = sbase + kOffP;
    float* s_sum = reinterpret_cast<float*>(smem + kOffKV) + 2 * g * kBM + row;  // [half][row]
    if (ok) s_sum[half * kBM] = l;
    pair_sync();
    if (ok) l += s_sum[(half ^ 1) * kBM];
    if constexpr (kSplit) {
      // The parts' references and sums are exchanged; then every row is scaled for the common ones and goes to the CTA
      // that adds up its parts, in their order: rows_own of the 256 rows each. Q, P and the ring are idle in every CTA
      // by then, and the rows arrive where Q and P were.
      const int rows_own = 2 * kBM / parts, ri = g * kBM + row;
      const uint32_t ml = sbase + kOffKV + 4 * kBM * 4;  // behind the halves' sums of 256 rows
      float ref = by_maximum ? m : 0.f;
      if (!ok || n_tiles == 0) {
        ref = -INFINITY;
        l = 0.f;
      }
      if (half == 0) asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ml + ri * 8), "f"(ref), "f"(l) : "memory");
      cluster_sync();
      float M = -INFINITY, L = 0.f;
      for (int i = 0; i < parts; ++i) M = fmaxf(M, ld_cluster_f2(in_part(ml + ri * 8, i)).x);
      if (M == -INFINITY) M = 0.f;
      for (int i = 0; i < parts; ++i) {
        const float2 v = ld_cluster_f2(in_part(ml + ri * 8, i));
        L = fmaf(ex2_approx(v.x - M), v.y, L);
      }
      const float inv = ex2_approx(ref - M) * (L == 0.f ? 0.f : 1.f / L);
      const uint32_t dst = in_part(sbase + kOffQ + (part * rows_own + ri % rows_own) * 512, ri / rows_own);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) {
        uint32_t x[32];
        if (ok && n_tiles > 0) {
          tmem_ld32(tO + c * 32, x);
          tmem_wait_ld();
          tmem_reg_fence(x);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          st_cluster_f4(dst + (((half * 16 + c * 8 + j / 4) ^ (row & 31)) << 4), __uint_as_float(x[j]) * inv,
                        __uint_as_float(x[j + 1]) * inv, __uint_as_float(x[j + 2]) * inv, __uint_as_float(x[j + 3]) * inv);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarStaged));
      cluster_sync();
      for (int lr = warp - 4; lr < rows_own; lr += kSoftmaxWarps) {
        const int r2 = part * rows_own + lr, g2 = r2 / kBM, q_row = r2 % kBM;
        const int seq_row = r0 + q_row + (p.neighbours ? g2 * kBM : 0), to_head = head0 + (p.neighbours ? 0 : g2);
        if (seq_row >= Lq) continue;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < parts; ++i) {
          float4 v;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                       : "r"(sbase + kOffQ + (i * rows_own + lr) * 512 + ((lane ^ (q_row & 31)) << 4))
                       : "memory");
          o.x += v.x;
          o.y += v.y;
          o.z += v.z;
          o.w += v.w;
        }
        const int64_t out_row = static_cast<int64_t>(cq0) + seq_row;
        if (__any_sync(0xffffffffu, isnan(fmaf(o.x, 0.f, fmaf(o.y, 0.f, fmaf(o.z, 0.f, o.w * 0.f)))))) {
          int row_pos, row_lo, row_hi;
          seen_from(seq_row, row_pos, row_lo, row_hi);
          row_again<E>(p, b, ck0, out_row, to_head, row_pos, row_lo, row_hi, lane);
        } else {
          *(reinterpret_cast<uint2*>(p.out + (out_row * p.hq + to_head) * kHeadDim) + lane) =
              make_uint2(Ops::pack(o.x, o.y), Ops::pack(o.z, o.w));
        }
      }
      wait_for_others();
      return;
    }
    if (ok) {
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float spoilt = 0.f;  // NaN once any element is not finite
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(tO + c * 32, r);
        tmem_wait_ld();
        tmem_reg_fence(r);
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          const int q = g * 16 + half * 8 + c * 4 + j / 8;  // 16-byte chunk of the 512-byte row
          sts128(stage + row * 512 + ((q ^ (row & 31)) << 4),
                 Ops::pack(__uint_as_float(r[j + 0]) * inv, __uint_as_float(r[j + 1]) * inv),
                 Ops::pack(__uint_as_float(r[j + 2]) * inv, __uint_as_float(r[j + 3]) * inv),
                 Ops::pack(__uint_as_float(r[j + 4]) * inv, __uint_as_float(r[j + 5]) * inv),
                 Ops::pack(__uint_as_float(r[j + 6]) * inv, __uint_as_float(r[j + 7]) * inv));
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) spoilt = fmaf(__uint_as_float(r[j]), 0.f, spoilt);
      }
      const uint32_t again = __ballot_sync(0xffffffffu, isnan(spoilt) && g_row0 + row < Lq);
      if (lane == 0 && again) atomicOr(s_again + rows32, again);
    }
    // all softmax warps arrive, whatever happened, so the wait below (and
    // warp 1's before releasing TMEM) always ends; every tensor-memory read of
    // this warp is complete here
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarStaged));
    const bool staged = __all_sync(0xffffffffu, wait_or_abort(bar(kBarStaged), 0, s_abort, p.err));
    if (ok && staged) {
      const int to_g = lane >> 4;  // this lane's half of the 512 bytes
      const int to_row0 = r0 + (p.neighbours ? to_g * kBM : 0);
      uint16_t* obase = p.out + (static_cast<int64_t>(cq0 + to_row0) * p.hq + head0 + (p.neighbours ? 0 : to_g)) * kHeadDim +
                        (lane & 15) * 8;
      const uint32_t* skip = s_again + 4 * to_g;
      for (int rr = warp - 4; rr < min(kBM, Lq - r0); rr += kSoftmaxWarps) {
        uint32_t a, b2, c2, d;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a), "=r"(b2), "=r"(c2), "=r"(d)
                     : "r"(stage + rr * 512 + ((lane ^ (rr & 31)) << 4)));
        if (to_row0 + rr < Lq && !((skip[rr >> 5] >> (rr & 31)) & 1u))
          *reinterpret_cast<uint4*>(obase + static_cast<int64_t>(rr) * p.hq * kHeadDim) = make_uint4(a, b2, c2, d);
      }
      for (uint32_t again = half == 0 ? s_again[rows32] : 0; again; again &= again - 1) {
        const int src = __ffs(again) - 1;
        row_again<E>(p, b, ck0, static_cast<int64_t>(cq0) + g_row0 + (warp & 3) * 32 + src, head,
                     __shfl_sync(0xffffffffu, pos, src), __shfl_sync(0xffffffffu, lo, src),
                     __shfl_sync(0xffffffffu, hi, src), lane);
      }
    }
  }

  if (kSplit) {  // (warps 0 to 3 here) every thread of a cluster comes to both of its barriers
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    // TMEM is released after every softmax warp's last tensor-memory read
    // (they all arrive on kBarStaged once O is staged); no CTA-wide barrier,
    // so no role waits at one with some of its lanes still busy. The wait is
    // time-bounded but ignores the abort flag: the softmax warps always arrive.
    __syncwarp();
    mbar_wait(bar(kBarStaged), 0, p.err);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (kSplit) {
    cluster_sync();
    wait_for_others();
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                                        &q) == cudaSuccess && q == cudaDriverEntryPointSuccess;
    return found ? reinterpret_cast<EncodeTiledFn>(ptr) : nullptr;
  }();
  return fn;
}

// [rows, heads, 128] view of 16-bit elements with rows row_stride_elems apart;
// box = 128 rows x 1 head x 64 dims.
bool encode_rows_heads_dims(CUtensorMap* tm, const void* base, int64_t rows, int heads, int64_t row_stride_elems,
                            Elem elem) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim * 2),
                                 static_cast<cuuint64_t>(row_stride_elems * 2)};
  const cuuint32_t box[3] = {64, 1, 128};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = elem == Elem::kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(tm, dt, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DeviceLimits {
  bool known;
  int sms;
  int clusters[4];  // [i], i > 0: clusters of 2^i CTAs that run at once
};

template <Elem E, bool kCap, bool kBias>
cudaError_t device_limits(DeviceLimits* out) {
  static DeviceLimits all[64];
  static std::mutex lock;
  const std::lock_guard<std::mutex> hold(lock);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && all[dev].known) {
    *out = all[dev];
    return cudaSuccess;
  }
  DeviceLimits d{};
  e = cudaFuncSetAttribute(prefill_mod_kernel<E, kCap, kBias, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemBytes));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(prefill_mod_kernel<E, kCap, kBias, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes));
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  for (int i = 1; i < 4 && e == cudaSuccess; ++i) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(d.sms) << i);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << i;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&d.clusters[i], prefill_mod_kernel<E, kCap, kBias, true>, &cfg);
  }
  if (e != cudaSuccess) return e;
  d.known = true;
  if (dev >= 0 && dev < 64) all[dev] = d;
  *out = d;
  return cudaSuccess;
}

// The items run longest first, one CTA to an SM. What is left of them after whole rounds would keep a few SMs busy for one
// more item, and a call of few items uses few SMs from the start. Where all of that rest can run at once with each item's
// keys split over a cluster of 2, 4 or 8 CTAs, it does, as a launch of its own that fills SMs as the first one leaves
// them, the most parts first that leave a part kMinPartTiles key tiles. Times in key tiles (about 1.9 us each), as far as
// the bounds of the lengths tell them: the rest takes `tiles` as it is, less what it fits into the first round's uneven
// end (after an even number of rounds the long and the short items have evened out), and tiles / parts when split, plus
// 2 for the join and 2 for the launch beside others.
constexpr int kMinPartTiles = 2;
template <Elem E, bool kCap, bool kBias>
cudaError_t launch_typed(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, PrefillModParams& p,
                         int64_t n_items, int64_t max_tiles, int64_t seen_tiles, cudaStream_t stream) {
  DeviceLimits d;
  cudaError_t e = device_limits<E, kCap, kBias>(&d);
  if (e != cudaSuccess) return e;
  const int64_t rest = n_items % d.sms, rounds = n_items / d.sms;
  int shift = 0;
  if (rest > 0) {
    const int64_t per_tile = static_cast<int64_t>(p.num_seqs) * p.units;  // items as long as one another
    const int64_t shorter = (n_items - rest) / per_tile * (p.neighbours ? 2 : 1);
    const int64_t tiles = std::min(max_tiles - shorter, seen_tiles);  // key tiles of the first of the rest
    const int64_t uneven = rounds % 2 == 1 ? d.sms / per_tile : 0;
    for (int i = 1; i < 4; ++i) {
      const int64_t split = (tiles >> i) + (rounds > 0 ? 4 : 2);
      if (rest <= d.clusters[i] && tiles >> i >= kMinPartTiles && tiles - uneven - split >= 2) shift = i;
    }
  }
  const int64_t whole = shift > 0 ? n_items - rest : n_items;
  p.first = 0;
  if (whole > 0) {
    prefill_mod_kernel<E, kCap, kBias, false><<<static_cast<unsigned>(whole), kThreads, kSmemBytes, stream>>>(tq, tk, tv, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (shift == 0) return cudaSuccess;
  p.first = static_cast<int32_t>(whole);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rest) << shift);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1u << shift;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = whole > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, prefill_mod_kernel<E, kCap, kBias, true>, tq, tk, tv,
                            const_cast<const PrefillModParams&>(p));
}

template <Elem E>
cudaError_t launch_elem(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, PrefillModParams& p,
                        int64_t n_items, int64_t max_tiles, int64_t seen_tiles, cudaStream_t stream) {
  if (p.softcap > 0.f)
    return p.slopes ? launch_typed<E, true, true>(tq, tk, tv, p, n_items, max_tiles, seen_tiles, stream)
                    : launch_typed<E, true, false>(tq, tk, tv, p, n_items, max_tiles, seen_tiles, stream);
  return p.slopes ? launch_typed<E, false, true>(tq, tk, tv, p, n_items, max_tiles, seen_tiles, stream)
                  : launch_typed<E, false, false>(tq, tk, tv, p, n_items, max_tiles, seen_tiles, stream);
}

// z = sum over i of scale_log2 c_i c^2i (q.k)^(2i + 1), c = scale / cap. Where the powers of c leave fp32's range (odd
// scales, far from any use) the first polynomial is kept to |x| <= 0.02 cap, where its last terms are nothing, and the
// second is not used.
template <Elem E>
void fit_tanh(PrefillModParams& p) {
  using Fit = TanhFit<E>;
  const double c = static_cast<double>(p.scale) / p.softcap, s = static_cast<double>(p.scale) * 1.4426950408889634;
  for (int i = 0; i < 6; ++i) {
    // (c >= 100: nothing but zeros goes through them, and stays zero)
    p.near_c[i] = c < 100 || i == 0 ? static_cast<float>(s * Fit::kNearC[i] * std::pow(c, 2 * i)) : 0.f;
    p.far_c[i] = c < 100 || i == 0 ? static_cast<float>(s * Fit::kFarC[i] * std::pow(c, 2 * i)) : 0.f;
    p.tanh_c[i] = static_cast<float>(Fit::kFarC[i]);
  }
  p.near_top = c < 100 ? static_cast<float>(std::fmin((c > 1e-5 ? Fit::kNearTop : 0.02) / c, 1e18)) : 0.f;
  p.far_top = c < 100 && c > 1e-3 ? static_cast<float>(Fit::kFarTop / c) : 0.f;
}

cudaError_t launch_prefill_mod(const PrefillModArgs& a, unsigned int* err, cudaStream_t stream, Elem elem) {
  const bool paged = a.block_tables != nullptr;
  const int64_t kv_rows = paged ? static_cast<int64_t>(a.num_blocks) * kBlockSize : a.total_k;
  const int64_t kv_stride = paged ? static_cast<int64_t>(a.hkv) * kHeadDim : a.kv_row_stride;
  CUtensorMap tq, tk, tv;
  if (!encode_rows_heads_dims(&tq, a.q, a.total_q, a.hq, a.q_row_stride, elem) ||
      !encode_rows_heads_dims(&tk, a.k, kv_rows, a.hkv, kv_stride, elem) ||
      !encode_rows_heads_dims(&tv, a.v, kv_rows, a.hkv, kv_stride, elem))
    return cudaErrorInvalidValue;
  PrefillModParams p{};
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.block_tables = a.block_tables;
  p.bt_stride = a.bt_stride;
  p.num_blocks = a.num_blocks;
  p.num_seqs = a.num_seqs;
  p.hq = a.hq;
  p.group = a.hq / a.hkv;
  p.neighbours = p.group % 2;
  p.units = p.neighbours ? a.hq : a.hq / 2;
  const int rows = p.neighbours ? 2 * kBM : kBM;
  p.q_tiles = static_cast<int32_t>((static_cast<int64_t>(std::min(a.max_seqlen_q, a.total_q)) + rows - 1) / rows);
  p.max_seqlen_q = a.max_seqlen_q;
  p.max_seqlen_k = a.max_seqlen_k;
  p.total_q = a.total_q;
  p.total_k = paged ? 0 : a.total_k;
  p.paged = paged ? 1 : 0;
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  p.softcap = a.softcap < kNoCap ? a.softcap : 0.f;
  if (p.softcap > 0.f) {
    p.cap_log2 = p.softcap * kLog2e;
    p.scale_by_cap = fminf(a.scale / p.softcap, FLT_MAX);  // not infinity: a score of 0 stays 0
    elem == Elem::kF16 ? fit_tanh<Elem::kF16>(p) : fit_tanh<Elem::kBF16>(p);
    p.fixed = elem == Elem::kBF16 && p.softcap <= kFixedCap;
  }
  p.slopes = a.slopes;
  p.window = a.window;
  p.key_starts = a.key_starts;
  p.prefix_lens = a.prefix_lens;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.q_stride = a.q_row_stride;
  p.kv_stride = kv_stride;
  p.out = static_cast<uint16_t*>(a.out);
  p.err = err;
  const int64_t n_items = static_cast<int64_t>(p.q_tiles) * a.num_seqs * p.units;
  if (n_items > 0x7fffffff) return cudaErrorInvalidValue;
  // key tiles of the last query tile at most
  int64_t keys = a.max_seqlen_k;
  if (paged) keys = std::min(keys, static_cast<int64_t>(a.bt_stride) * kBlockSize);
  const int64_t max_tiles = (keys + kBN - 1) / kBN;
  const int64_t seen_tiles = a.window > 0 && !a.prefix_lens ? (static_cast<int64_t>(a.window) + rows) / kBN + 1 : max_tiles;
  return elem == Elem::kF16 ? launch_elem<Elem::kF16>(tq, tk, tv, p, n_items, max_tiles, seen_tiles, stream)
                            : launch_elem<Elem::kBF16>(tq, tk, tv, p, n_items, max_tiles, seen_tiles, stream);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int prefill_mod_common(const void* q, int64_t q_row_stride, int32_t total_q, const void* k, const void* v,
                       int64_t kv_row_stride, int32_t total_k, const void* k_cache, const void* v_cache,
                       int32_t num_blocks, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                       int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* block_tables,
                       int32_t block_table_stride, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                       int32_t head_dim, int32_t block_size, float softmax_scale, float softcap, const float* slopes,
                       int32_t window, const int32_t* key_starts, const int32_t* prefix_lens, void* out,
                       cudaStream_t stream, Elem elem) {
  if (head_dim != kHeadDim || block_size != kBlockSize || num_kv_heads <= 0 || num_heads <= 0 || num_heads > 8192 ||
      num_heads % num_kv_heads != 0)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs < 0 || num_seqs > 65535 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 ||
      max_seqlen_q > (1 << 24) || max_seqlen_k > (1 << 24) || window < 0)
    return PKV_ERR_BAD_SIZE;
  if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return PKV_OK;
  if (!(softmax_scale > 0.f) || std::isinf(softmax_scale) || !(softcap >= 0.f) || std::isinf(softcap))
    return PKV_ERR_BAD_SIZE;
  if (!q || !out || !cu_seqlens_q || !cu_seqlens_k) return PKV_ERR_NULL_POINTER;
  const bool paged = block_tables != nullptr;
  const void* keys = paged ? k_cache : k;
  const void* values = paged ? v_cache : v;
  if (!keys || !values) return PKV_ERR_NULL_POINTER;
  if (paged ? num_blocks <= 0 || num_blocks > (1 << 23) - 1 || block_table_stride <= 0 : total_k == 0)
    return PKV_ERR_BAD_SIZE;
  if (q_row_stride < static_cast<int64_t>(num_heads) * head_dim ||
      (!paged && kv_row_stride < static_cast<int64_t>(num_kv_heads) * head_dim))
    return PKV_ERR_BAD_STRIDE;
  if (!aligned(q, 16) || q_row_stride % 8 != 0 || !aligned(out, 16) || !aligned(keys, 16) || !aligned(values, 16) ||
      (!paged && kv_row_stride % 8 != 0) || !aligned(slopes, 4) || !aligned(key_starts, 4) || !aligned(prefix_lens, 4))
    return PKV_ERR_ALIGNMENT;
  unsigned int* err = nullptr;
  const int st = device_error_word(&err);
  if (st != PKV_OK) return st;
  const PrefillModArgs a{q,          q_row_stride, total_q,      keys,         values,       kv_row_stride,
                         total_k,    num_blocks,   cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                         block_tables, block_table_stride, num_seqs, num_heads, num_kv_heads, softmax_scale,
                         softcap,    slopes,       window,       key_starts,   prefix_lens,  out};
  if (launch_prefill_mod(a, err, stream, elem) == cudaSuccess) return PKV_OK;
  (void)cudaGetLastError();
  return PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" {

// The bf16 and fp16 entry points share one body; only the elements' type differs.

int pkv_prefill_varlen_mod(const void* q, int64_t q_row_stride, int32_t total_q, const void* k, const void* v,
                           int64_t kv_row_stride, int32_t total_k, const void* k_cache, const void* v_cache,
                           int32_t num_blocks, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                           int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* block_tables,
                           int32_t block_table_stride, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                           int32_t head_dim, int32_t block_size, float softmax_scale, float softcap,
                           const float* slopes, int32_t window, const int32_t* key_starts, const int32_t* prefix_lens,
                           void* out, cudaStream_t stream) {
  return pkv::prefill_mod_common(q, q_row_stride, total_q, k, v, kv_row_stride, total_k, k_cache, v_cache, num_blocks,
                                 cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, block_tables,
                                 block_table_stride, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                 softmax_scale, softcap, slopes, window, key_starts, prefix_lens, out, stream,
                                 pkv::Elem::kBF16);
}

int pkv_prefill_varlen_mod_f16(const void* q, int64_t q_row_stride, int32_t total_q, const void* k, const void* v,
                               int64_t kv_row_stride, int32_t total_k, const void* k_cache, const void* v_cache,
                               int32_t num_blocks, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                               int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* block_tables,
                               int32_t block_table_stride, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                               int32_t head_dim, int32_t block_size, float softmax_scale, float softcap,
                               const float* slopes, int32_t window, const int32_t* key_starts,
                               const int32_t* prefix_lens, void* out, cudaStream_t stream) {
  return pkv::prefill_mod_common(q, q_row_stride, total_q, k, v, kv_row_stride, total_k, k_cache, v_cache, num_blocks,
                                 cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, block_tables,
                                 block_table_stride, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                 softmax_scale, softcap, slopes, window, key_starts, prefix_lens, out, stream,
                                 pkv::Elem::kF16);
}

}  // extern "C"
