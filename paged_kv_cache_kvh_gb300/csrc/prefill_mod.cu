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
// A CTA goes from item to item, taking the next from the launch's CTAs that have not begun (cluster launch control) when
// the last loads of its item are under way: whoever is done first gets the longest of what is left, and the next item's
// queries, keys and first products run under the last tile and the end of this one (16 k rows of 100..1024-token prompts
// with a cap and a window 77 us with a CTA to an item, 68 now; 5000 on 7001 without a cap 311 and 322, see Place).
//
// What bounds it: a key tile of both groups takes about 2 us, its products 1.1 of that; the rest is the chain of each
// group (product, softmax, barrier, product) with two groups to overlap: the tensor pipe is 54 % in use and the issue
// slots 49 %. 16 on 8 heads, 5000 on 7001 in the cache: 350 us capped at 50 and 322 without a cap, of 207 at
// cuBLAS' rate (0.59 and 0.64 of it). Measured and not kept: 384 threads with registers shared out by role (427 us where
// 404 was), scores fetched a tile ahead (430: three slots of the ring are too few for it).
//
// tanh: the softmax is issue-limited, and tanh through exponential and reciprocal would triple its special function
// work (128 x 128 scores a group: 2 us a tile of 1.6). An odd polynomial on packed pairs costs 4 instructions a pair for
// bf16 where all of a warp's |x| <= 0.4 cap, 6 up to the cap (fp16: one more each); only a tile with scores beyond goes
// through 1 - 2 / (1 + e^2x). A score is off by at most 7e-6 of itself for bf16 (p by 2^-12 at a score of 32, where its
// rounding to 16 bits loses 2^-9) and 6e-7 for fp16 (2^-15; 2^-12).
//
// The maximum: rows go by a reference (of fp16 rows 2^7 below the largest score, see kLift) that is moved when a score
// passes it by 2^8 and subtracted where the scores are scaled, so a tile needs one pass for the largest value and nothing
// else. Scores of bf16 rows capped at 52 or less need none at all: 2^z lies within 2^-75 .. 2^75, sums of it times v within
// fp32 (|v| up to 2^52; beyond, the row is computed again, see below), and bf16 keeps the same relative precision there as
// near 1.
//
// Values of V at keys that a row does not see are multiplied by p = 0; where they are not finite the sum is spoilt
// (0 * NaN). The rows of V behind the sequence's end, which may hold anything, are zeroed in shared memory. Elsewhere
// such values are rare, so they are found in the result: a row whose sum is not finite, and whose visible keys do not
// account for that, is computed once more by a warp that has nothing else to do, from the rows in memory, one key to a lane,
// with the keys that it does not see left out (one NaN behind 5000 cached keys, 12,800 rows of 2 heads: 1.1 ms where all
// rows but a tile's see it, 130 where 254 of one tile do not, 0.3 without it).
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
constexpr int kBarVTail = kBarOFinal + 1;         // +item % 2: zeros are behind the last value
constexpr int kBarDrain = kBarVTail + 2;
constexpr int kBarDone = kBarDrain + 1;           // the softmax warps have read tensor memory for the last time
constexpr int kBarItemFull = kBarDone + 1;        // +item % 2: it is described
constexpr int kBarItemFree = kBarItemFull + 2;    // +item % 2: everyone has read its description
constexpr int kBarQFree = kBarItemFree + 2;       // an item's last product with Q is complete
constexpr int kBarOFree = kBarQFree + 1;          // +group: its O has been read
constexpr int kBarNext = kBarOFree + 2;           // the next item's number has arrived
constexpr int kBarRows = kBarNext + 1;            // +item % 2: its rows have been written
constexpr int kNumBars = kBarRows + 2;
constexpr int kOffNext = kOffBar + (kNumBars * 8 + 15) / 16 * 16;  // where the hardware writes it, 16 bytes
constexpr int kOffItems = kOffNext + 16;

// What the roles of a CTA have to know of an item.
struct Item {
  int32_t b, head0, cq0, ck0, Lq, Lk;
  int32_t r0;              // first query row
  int32_t tile0, n_tiles;  // key tiles; n_tiles < 0: no more items
};
constexpr int kOffAgain = kOffItems + 2 * sizeof(Item);  // [item % 2][32 rows][half] rows to be computed again
constexpr int kOffSeen = (kOffAgain + 2 * kSoftmaxWarps * 4 + 15) / 16 * 16;  // [warp] the keys that any and that all of its rows see
constexpr int kOffMisc = kOffSeen + kSoftmaxWarps * 16;  // tmem address, abort flag, when rows were last computed again
constexpr size_t kSmemBytes = kOffMisc + 16 + 1024;      // + alignment slack
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
// A row's largest share before it is divided by their sum, log2: fp16 shares go down to 2^-24 in steps of as much, so those
// from 2^-21 of the largest on keep 11 bits (and 2^7 with 2^8 of headroom stays below fp16's largest number).
template <Elem E>
constexpr float kLift = E == Elem::kF16 ? 7.f : 0.f;
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
//
// Rows that are computed again may take longer than the limit (one value that is not finite, before long ranges of keys),
// and the waits for an item's description, and for the last reader of an older one, wait for them in the end. There
// (kBehindRows) the limit counts from when those rows last went on, if that is later than the wait's begin.
__device__ __forceinline__ volatile uint64_t* rows_went_on(volatile int* abort_flag) {
  return reinterpret_cast<volatile uint64_t*>(abort_flag + 1);
}
template <bool kBehindRows = false>
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                              unsigned int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      if (kBehindRows) {
        const uint64_t went_on = *rows_went_on(abort_flag);  // read before the time that it is taken from
        if (globaltimer_ns() - went_on <= kWaitLimitNs) continue;
      }
      flag_error(err, PKV_DEVERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_for_item(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
  return wait_or_abort<true>(bar, parity, abort_flag, err);
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

// Row r of an item's sequence: its position and the keys it sees. Rows behind the last one take its place.
__device__ __forceinline__ void seen_from(const PrefillModParams& p, const Item& it, int r, int& pos, int& lo, int& hi) {
  r = min(r, it.Lq - 1);
  pos = it.Lk - it.Lq + r;
  lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  if (p.key_starts) lo = max(lo, p.key_starts[it.cq0 + r]);
  hi = min(it.Lk, max(pos + 1, p.prefix_lens ? p.prefix_lens[it.b] : 0));
}

// The elements of a key's row of K or V, from the first of kv head hk's.
__device__ __forceinline__ int64_t key_place(const PrefillModParams& p, int b, int64_t k0, int hk, int t) {
  if (!p.paged) return (k0 + t) * p.kv_stride + hk * kHeadDim;
  int blk = p.block_tables[static_cast<int64_t>(b) * p.bt_stride + t / kBlockSize];
  if (blk < 0 || blk >= p.num_blocks) blk = 0;  // reported where the tile was fetched
  return (static_cast<int64_t>(blk) * kBlockSize + t % kBlockSize) * p.kv_stride + hk * kHeadDim;
}

// One (row of the item's sequence, query head) by a whole warp from the rows in memory: a key to a lane, then four dims to a
// lane; eight rows of V on the way (32 keys 3.2 us; one row of V at a time 26).
template <Elem E>
__device__ __forceinline__ void row_again(const PrefillModParams& p, const Item& it, int head, int row,
                                          volatile uint64_t* went_on) {
  using Ops = ElemOps<E>;
  const int lane = threadIdx.x & 31, hk = head / p.group;
  const int64_t at = static_cast<int64_t>(it.cq0) + row;
  const uint4* q = reinterpret_cast<const uint4*>(p.q + at * p.q_stride + head * kHeadDim);
  const float slope = p.slopes ? p.slopes[head] * kLog2e : 0.f;
  int pos, lo, hi;
  seen_from(p, it, row, pos, lo, hi);
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};  // l: of this lane's keys
  for (int t0 = lo < hi ? lo & ~31 : hi; t0 < hi; t0 += 32) {
    if (lane == 0 && (t0 & 1023) == 0) *went_on = globaltimer_ns();
    const int64_t place = key_place(p, it.b, it.ck0, hk, t0);  // 32 keys lie in one block
    const int t = t0 + lane;
    const bool seen = t >= lo && t < hi;
    float z = -INFINITY;
    if (seen) {
      const uint4* kr = reinterpret_cast<const uint4*>(p.k + place + lane * p.kv_stride);
      float x = 0.f;
#pragma unroll 4
      for (int i = 0; i < kHeadDim / 8; ++i) {
        const uint4 a = kr[i], c = q[i];
        x = fmaf(Ops::lo(a.x), Ops::lo(c.x), fmaf(Ops::hi(a.x), Ops::hi(c.x), x));
        x = fmaf(Ops::lo(a.y), Ops::lo(c.y), fmaf(Ops::hi(a.y), Ops::hi(c.y), x));
        x = fmaf(Ops::lo(a.z), Ops::lo(c.z), fmaf(Ops::hi(a.z), Ops::hi(c.z), x));
        x = fmaf(Ops::lo(a.w), Ops::lo(c.w), fmaf(Ops::hi(a.w), Ops::hi(c.w), x));
      }
      z = p.softcap > 0.f ? p.cap_log2 * tanhf(x * p.scale_by_cap) : x * p.scale_log2;
      z = fmaf(-slope, fabsf(static_cast<float>(pos - t)), z);
    }
    float top = fmaxf(m, z);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float use = top == -INFINITY ? 0.f : top;
    const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - use);
    const float e = seen ? ex2_approx(z - use) : 0.f;
    m = top;
    l = l * alpha + e;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= alpha;
    const uint16_t* vr = p.v + place + lane * 4;
    const int end = min(32, hi - t0);  // 0 times what is not finite must not be added: keys that are seen, and no others
#pragma unroll 8
    for (int i = max(0, lo - t0); i < end; ++i) {
      const float pi = __shfl_sync(0xffffffffu, e, i);
      const uint2 x = *reinterpret_cast<const uint2*>(vr + i * p.kv_stride);
      acc[0] = fmaf(pi, Ops::lo(x.x), acc[0]);
      acc[1] = fmaf(pi, Ops::hi(x.x), acc[1]);
      acc[2] = fmaf(pi, Ops::lo(x.y), acc[2]);
      acc[3] = fmaf(pi, Ops::hi(x.y), acc[3]);
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *(reinterpret_cast<uint2*>(p.out + (at * p.hq + head) * kHeadDim) + lane) =
      make_uint2(Ops::pack(acc[0] * inv, acc[1] * inv), Ops::pack(acc[2] * inv, acc[3] * inv));
}

// An item's marked rows, [group][half][32 rows]: those whose sums are not finite, though their shares are. That may come
// from keys that they see, and is right then: NaN where one of these is NaN; infinity where one is infinite, since any key
// that is not seen would have made it NaN. Such rows' marks are taken off; the others (values that a tile's products took in
// without being seen, sums beyond fp32) are to be computed again. What is known of the item's values, per dim, four to a
// lane: the first and the last key with NaN (infinity), and in which of up to 32 stretches of keys there is one.
template <Elem E>
__device__ __forceinline__ void settle_marks(const PrefillModParams& p, const Item& it, volatile uint32_t* marks,
                                             volatile uint64_t* went_on) {
  constexpr uint32_t kInf = E == Elem::kBF16 ? 0x7f80u : 0x7c00u;
  constexpr uint32_t kAdd = (0x8000u - kInf) * 0x10001u;  // carries into the sign's place from an exponent of ones
  const int lane = threadIdx.x & 31, hk = it.head0 / p.group;
  const int from = it.tile0 * kBN, to = min(it.Lk, from + it.n_tiles * kBN);
  const int stretch = ((to - from + 511) / 512) * 16;
  int first[2][4], last[2][4];  // [infinity][dim]
  uint32_t has[2][4];
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    first[d >> 2][d & 3] = INT32_MAX;
    last[d >> 2][d & 3] = -1;
    has[d >> 2][d & 3] = 0u;
  }
  for (int t0 = from; t0 < to; t0 += 16) {
    if (lane == 0 && (t0 & 1023) == 0) *went_on = globaltimer_ns();
    const uint16_t* vr = p.v + key_place(p, it.b, it.ck0, hk, t0) + lane * 4;
    uint2 x[16];
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      x[j] = t0 + j < to ? *reinterpret_cast<const uint2*>(vr + j * p.kv_stride) : make_uint2(0u, 0u);
#pragma unroll
    for (int j = 0; j < 16; ++j) any |= ((x[j].x & 0x7fff7fffu) + kAdd) | ((x[j].y & 0x7fff7fffu) + kAdd);
    if (!__any_sync(0xffffffffu, (any & 0x80008000u) != 0)) continue;
    const uint32_t bit = 1u << ((t0 - from) / stretch);
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t size = ((d < 2 ? x[j].x : x[j].y) >> (16 * (d & 1))) & 0x7fffu;
#pragma unroll
        for (int inf = 0; inf < 2; ++inf)
          if (inf ? size == kInf : size > kInf) {
            first[inf][d] = min(first[inf][d], t0 + j);
            last[inf][d] = t0 + j;
            has[inf][d] |= bit;
          }
      }
  }
  for (int i = 0; i < 8; ++i) {  // of 32 rows
    const int row0 = it.r0 + (i & 3) * 32 + (p.neighbours && i >= 4 ? kBM : 0);
    const int head = it.head0 + (p.neighbours ? 0 : i >> 2);
    volatile uint32_t* halves = marks + (i >> 2) * 8 + (i & 3);
    uint32_t again = halves[0] | halves[4];
    for (uint32_t left = again; left; left &= left - 1) {
      const int r = row0 + __ffs(left) - 1;
      int pos, lo, hi;
      seen_from(p, it, r, pos, lo, hi);
      // stretches that the row sees all of
      const int a = (max(lo - from, 0) + stretch - 1) / stretch, z = hi >= to ? 32 : (hi - from) / stretch;
      const uint32_t seen = a < z ? (0xffffffffu << a) & (0xffffffffu >> (32 - z)) : 0u;
      const int64_t at = (static_cast<int64_t>(it.cq0) + r) * p.hq + head;
      const uint2 o = *(reinterpret_cast<const uint2*>(p.out + at * kHeadDim) + lane);
      bool settled = true;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t size = ((d < 2 ? o.x : o.y) >> (16 * (d & 1))) & 0x7fffu;
#pragma unroll
        for (int inf = 0; inf < 2; ++inf)
          if (inf ? size == kInf : size > kInf)
            settled = settled && ((first[inf][d] >= lo && first[inf][d] < hi) || (last[inf][d] >= lo && last[inf][d] < hi) ||
                                  (has[inf][d] & seen) != 0);
      }
      if (__all_sync(0xffffffffu, settled)) again &= ~(left & -left);
    }
    __syncwarp();
    if (lane == 0) {
      halves[0] = again;
      halves[4] = 0;
    }
  }
  __syncwarp();
}

// What is left of an item's marked rows, by one warp. A function that finds its place in shared memory itself, one row at a
// time: other forms took registers from the kernel's loop over the tiles (four rows at once 93 instead of 142 ms for 254 rows
// of 5,100 keys, but any chunk of 5000 on 7001, capped, 367 us instead of 349).
template <Elem E>
__device__ __noinline__ void item_again(const PrefillModParams& p, int parity) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const Item& it = reinterpret_cast<const Item*>(smem + kOffItems)[parity];
  volatile uint32_t* marks = reinterpret_cast<volatile uint32_t*>(smem + kOffAgain) + parity * kSoftmaxWarps;
  volatile uint64_t* went_on = rows_went_on(reinterpret_cast<volatile int*>(smem + kOffMisc + 4));
  settle_marks<E>(p, it, marks, went_on);
  for (int i = 0; i < 8; ++i) {  // of 32 rows
    const int row0 = it.r0 + (i & 3) * 32 + (p.neighbours && i >= 4 ? kBM : 0);
    for (uint32_t again = marks[(i >> 2) * 8 + (i & 3)]; again; again &= again - 1)
      row_again<E>(p, it, it.head0 + (p.neighbours ? 0 : i >> 2), row0 + __ffs(again) - 1, went_on);
  }
}
template <Elem E>
__device__ __noinline__ void split_row_again(const PrefillModParams& p, const Item& it, int head, int row,
                                             volatile uint64_t* went_on) {
  row_again<E>(p, it, head, row, went_on);
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

// The next item, from the CTAs of the launch that have not begun yet: asks the hardware to cancel one of them and to write
// its place to `addr` (16 bytes, counted by the barrier). After an answer that there are none it must not be asked again.
__device__ __forceinline__ void ask_next(uint32_t addr, uint32_t bar) {
  fence_proxy_async_smem();  // the last answer has been read
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(addr),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool next_cta(uint32_t addr, int& cta) {
  uint32_t there, x = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 answer;\n\tld.shared.b128 answer, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, answer;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, answer;\n\t}"
      : "=r"(there), "=r"(x)
      : "r"(addr)
      : "memory");
  cta = static_cast<int>(x);
  return there != 0;
}

// A CTA goes from item to item, its roles one behind another: while the softmax warps finish an item, the next one's
// queries, keys and first products are under way. kSplit: the CTAs of a cluster have parts of one item's keys, and only
// that item.
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
  Item* items = reinterpret_cast<Item*>(smem + kOffItems);
  volatile uint32_t* s_again = reinterpret_cast<volatile uint32_t*>(smem + kOffAgain);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (!kSplit) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // items split over clusters fill the end
  const int parts = kSplit ? cluster_parts() : 1, part = kSplit ? cluster_part() : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      int count = 1;
      if (i == kBarPReady || i == kBarPReady + 1 || i == kBarOFree || i == kBarOFree + 1) count = kSoftmaxWarps / 2;
      if (i == kBarDone || i == kBarRows || i == kBarRows + 1) count = kSoftmaxWarps;
      if (i == kBarItemFree || i == kBarItemFree + 1) count = kSoftmaxWarps + 2;
      mbar_init(bar(i), count);
    }
    *s_abort = 0;
    *rows_went_on(s_abort) = 0;
    mbar_fence_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
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

  // Tile n of an item's: a bias favours the nearest keys: from the last tile to the first, the reference is found in the
  // first one and stays (5000 on 7001: 404 us from the first on, 331 from the last; without a bias 308 and 326).
  constexpr bool kBack = kBias;
  auto first_key_of = [&](const Item& it, int n) { return (it.tile0 + (kBack ? it.n_tiles - 1 - n : n)) * kBN; };
  // keys that the last of the tiles has, and the item's load of its values (the first load is 0)
  auto tail_of = [&](const Item& it) { return it.Lk - (it.tile0 + it.n_tiles - 1) * kBN; };
  auto tail_load = [&](const Item& it) { return kBack ? 1 : 2 * it.n_tiles - 1; };

  bool had_item = false;  // (kSplit, warps 0 to 3)
  if (warp == 0) {
    // =========================== items and their loads ===========================
    // Loads of all items are counted through: load x goes into slot x % kKvSlots.
    int ring = 0, k = 0;
    bool ok = true, waiting = false;  // for the next item's number, after an abort
    uint32_t next_parity = 0;
    int cta = static_cast<int>(blockIdx.x);
    const int per_tile = p.num_seqs * p.units;
    while (ok) {
      // ---- the last query tiles (the longest key ranges) first ----
      const int item = p.first + cta / parts;
      const int qt = p.q_tiles - 1 - item / per_tile, unit = item % p.units;
      Item it;
      it.b = (item % per_tile) / p.units;
      it.head0 = p.neighbours ? unit : 2 * unit;
      it.r0 = qt * (p.neighbours ? 2 * kBM : kBM);
      it.cq0 = p.cu_q[it.b];
      it.ck0 = p.cu_k[it.b];
      const int cq1 = p.cu_q[it.b + 1], ck1 = p.cu_k[it.b + 1];
      it.Lq = cq1 - it.cq0;
      it.Lk = ck1 - it.ck0;
      const bool bad = it.Lq < 0 || it.Lk < it.Lq || it.Lq > p.max_seqlen_q || it.Lk > p.max_seqlen_k || it.cq0 < 0 ||
                       cq1 > p.total_q || (p.paged ? it.Lk > static_cast<int64_t>(p.bt_stride) * kBlockSize
                                                   : (it.ck0 < 0 || ck1 > p.total_k));
      if (bad && lane == 0 && qt == 0 && unit == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
      if (!bad && it.r0 < it.Lq) {
        // the keys that any of the rows sees; a row that sees none widens nothing
        const int rows = p.neighbours ? 2 * kBM : kBM;
        int first_key = INT32_MAX, end_key = 0;
        for (int r = lane; r < (p.key_starts ? rows : 2); r += 32) {
          int pos, lo, hi;  // without first keys of single rows the first and the last row tell
          seen_from(p, it, p.key_starts ? it.r0 + r : (r == 0 ? it.r0 : it.r0 + rows - 1), pos, lo, hi);
          if (lo < hi) {
            first_key = min(first_key, lo);
            end_key = max(end_key, hi);
          }
        }
        first_key = __reduce_min_sync(0xffffffffu, first_key);
        end_key = __reduce_max_sync(0xffffffffu, end_key);
        // rows that see nothing at all: one tile, all masked
        const int all_tiles = first_key < end_key ? (end_key + kBN - 1) / kBN - first_key / kBN : 1;
        it.tile0 = (first_key < end_key ? first_key / kBN : 0) + (kSplit ? all_tiles * part / parts : 0);
        it.n_tiles = kSplit ? all_tiles * (part + 1) / parts - all_tiles * part / parts : all_tiles;  // 0 at times
        if (k >= 2) ok = __all_sync(0xffffffffu, wait_for_item(bar(kBarItemFree + (k & 1)), ((k >> 1) - 1) & 1, s_abort, p.err));
        if (!ok) break;
        if (lane == 0) {
          items[k & 1] = it;
          mbar_arrive(bar(kBarItemFull + (k & 1)));
        }
        had_item = true;
        if (k >= 1) ok = __all_sync(0xffffffffu, wait_or_abort(bar(kBarQFree), (k - 1) & 1, s_abort, p.err));
        if (!ok) break;
        const int hk = it.head0 / p.group;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(kBarQ), 2 * kTileBytes);
          for (int i = 0; i < 2; ++i) {
            const uint32_t dst = sbase + kOffQ + i * kTileBytes;
            const int head = it.head0 + (p.neighbours ? 0 : i), first = it.cq0 + it.r0 + (p.neighbours ? i * kBM : 0);
            tma_load_3d(dst, &tm_q, 0, head, first, bar(kBarQ));
            tma_load_3d(dst + kHalfBytes, &tm_q, 64, head, first, bar(kBarQ));
          }
        }
        int issued = 0;  // of the item's loads: K of tile i / 2 (even i) or V (odd i)
        auto issue_up_to = [&](int end) {
          if (lane == 0) {
            for (int i = issued; i < end; ++i) {
              const int x = ring + i, slot = x % kKvSlots;
              if (x >= kKvSlots && !wait_or_abort(bar(kBarKvFree + slot), ((x / kKvSlots) - 1) & 1, s_abort, p.err)) break;
              int at = first_key_of(it, i >> 1);
              if (p.paged) {
                int blk = p.block_tables[static_cast<int64_t>(it.b) * p.bt_stride + at / kBlockSize];
                if (blk < 0 || blk >= p.num_blocks) {
                  flag_error(p.err, PKV_DEVERR_BAD_BLOCK);
                  blk = 0;
                }
                at = blk * kBlockSize + at % kBlockSize;
              } else {
                at += it.ck0;
              }
              const CUtensorMap* tm = (i & 1) ? &tm_v : &tm_k;
              const uint32_t dst = sbase + kOffKV + slot * kTileBytes;
              mbar_arrive_expect_tx(bar(kBarKvFull + slot), kTileBytes);
              tma_load_3d(dst, tm, 0, hk, at, bar(kBarKvFull + slot));
              tma_load_3d(dst + kHalfBytes, tm, 64, hk, at, bar(kBarKvFull + slot));
              ++issued;
            }
          }
          issued = __shfl_sync(0xffffffffu, issued, 0);
        };
        const int tail_keys = tail_of(it), tail = tail_load(it);
        issue_up_to(kBack ? min(kKvSlots, 2 * it.n_tiles) : 2 * it.n_tiles);
        if (tail_keys < kBN && it.n_tiles > 0 && issued > tail) {
          // Zero the rows of the sequence's last V tile that lie past its end.
          const int slot = (ring + tail) % kKvSlots;
          if (wait_or_abort(bar(kBarKvFull + slot), ((ring + tail) / kKvSlots) & 1, s_abort, p.err)) {
            const uint32_t base = sbase + kOffKV + slot * kTileBytes;
            // rows tail_keys..127 of both 64-dim halves: 128-byte rows, swizzle
            // only permutes 16-byte chunks within a row.
            const int nz = (kBN - tail_keys) * 2 * 8;  // 16-byte chunks
            for (int c = lane; c < nz; c += 32) {
              const int at = tail_keys + (c >> 4), half = (c >> 3) & 1, chunk = c & 7;
              sts128(base + half * kHalfBytes + at * 128 + chunk * 16, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(bar(kBarVTail + (k & 1)));  // of every item
        issue_up_to(2 * it.n_tiles);
        ring += issued;
        ++k;
        ok = issued == 2 * it.n_tiles;
      }
      if (kSplit || !ok) break;
      // asked for when this item's last loads are under way, not before: whoever is done first has the longest of the rest
      if (lane == 0) ask_next(sbase + kOffNext, bar(kBarNext));
      if (!__all_sync(0xffffffffu, wait_or_abort(bar(kBarNext), next_parity, s_abort, p.err))) {
        waiting = true;
        break;
      }
      next_parity ^= 1;
      const bool there = next_cta(sbase + kOffNext, cta);
      __syncwarp();
      if (!there) break;
    }
    // no more items
    if (ok && k >= 2) ok = wait_for_item(bar(kBarItemFree + (k & 1)), ((k >> 1) - 1) & 1, s_abort, p.err);
    ok = __all_sync(0xffffffffu, ok);
    if (lane == 0) {
      if (ok) {
        items[k & 1].n_tiles = -1;
        mbar_arrive(bar(kBarItemFull + (k & 1)));
      }
      // Never leave a copy in flight into this CTA's shared memory.
      if (k > 0) mbar_wait(bar(kBarQ), (k - 1) & 1, p.err);
      for (int x = max(0, ring - kKvSlots); x < ring; ++x)
        mbar_wait(bar(kBarKvFull + x % kKvSlots), (x / kKvSlots) & 1, p.err);
      if (waiting) mbar_wait(bar(kBarNext), next_parity, p.err);
    }
  } else if (warp == 1) {
    // =========================== MMA issuer ===========================
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_f16kind_f32(kBM, kBN, false, false, Ops::kMmaFormat);
      constexpr uint32_t idesc_pv = idesc_f16kind_f32(kBM, kHeadDim, false, true, Ops::kMmaFormat);
      auto slot_of = [](int x) { return x % kKvSlots; };
      auto par_of = [](int x) { return static_cast<uint32_t>((x / kKvSlots) & 1); };
      // Descriptor low halves: each product below costs two 32-bit adds and
      // the tcgen05.mma (this one thread issues every product of the CTA).
      const uint32_t lo_kmaj = desc_lo(sbase, 16), lo_v = desc_lo(sbase, kHalfBytes);
      auto issue_s = [&](int i, int slot) {
        const uint32_t qa = lo_kmaj + ((kOffQ + i * kTileBytes) >> 4);
        const uint32_t kbb = lo_kmaj + (kOffKV >> 4) + slot * (kTileBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < kHeadDim / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
          mma_f16kind_lo(tmem + i * 128, qa + off, kbb + off, idesc_s, ks > 0 ? 1u : 0u);
        }
        mma_commit(bar(kBarSFull + i));
      };
      auto issue_pv = [&](int i, int slot, bool first) {
        const uint32_t pa = lo_kmaj + ((kOffP + i * kTileBytes) >> 4);
        const uint32_t vbb = lo_v + (kOffKV >> 4) + slot * (kTileBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < kBN / 16; ++ks) {
          const uint32_t aoff = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
          mma_f16kind_lo(tmem + 256 + i * 128, pa + aoff, vbb + ((ks * 16 * 128) >> 4), idesc_pv,
                         (!first || ks > 0) ? 1u : 0u);
        }
      };
      int ring = 0, t = 0;  // loads and tiles of the items before
      bool ok = true;
      for (int k = 0;; ++k) {
        if (!(ok = wait_for_item(bar(kBarItemFull + (k & 1)), (k >> 1) & 1, s_abort, p.err))) break;
        const Item it = items[k & 1];
        if (it.n_tiles < 0) break;
        had_item = true;
        mbar_arrive(bar(kBarItemFree + (k & 1)));
        if (!(ok = wait_or_abort(bar(kBarQ), k & 1, s_abort, p.err))) break;
        const bool v_tail = tail_of(it) < kBN && it.n_tiles > 0;
        if (it.n_tiles > 0) {
          if (!(ok = wait_or_abort(bar(kBarKvFull + slot_of(ring)), par_of(ring), s_abort, p.err))) break;
          tc_fence_after();
          issue_s(0, slot_of(ring));
          issue_s(1, slot_of(ring));
          mma_commit(bar(kBarKvFree + slot_of(ring)));
          if (it.n_tiles == 1) mma_commit(bar(kBarQFree));
        }
        for (int n = 0; n < it.n_tiles; ++n) {
          const int xv = ring + 2 * n + 1, xk = xv + 1;
          if (v_tail && 2 * n + 1 == tail_load(it))
            ok = wait_or_abort(bar(kBarVTail + (k & 1)), (k >> 1) & 1, s_abort, p.err);
          else
            ok = wait_or_abort(bar(kBarKvFull + slot_of(xv)), par_of(xv), s_abort, p.err);
          if (!ok) break;
          const bool more = n + 1 < it.n_tiles;
          for (int i = 0; ok && i < 2; ++i) {
            if (!(ok = wait_or_abort(bar(kBarPReady + i), (t + n) & 1, s_abort, p.err))) break;
            if (n == 0 && k > 0 && !(ok = wait_or_abort(bar(kBarOFree + i), (k - 1) & 1, s_abort, p.err))) break;
            tc_fence_after();
            issue_pv(i, slot_of(xv), n == 0);
            if (i == 1) mma_commit(bar(kBarKvFree + slot_of(xv)));
            if (!more) continue;
            if (i == 0) {
              if (!(ok = wait_or_abort(bar(kBarKvFull + slot_of(xk)), par_of(xk), s_abort, p.err))) break;
              tc_fence_after();
            }
            issue_s(i, slot_of(xk));
            if (i == 1) {
              mma_commit(bar(kBarKvFree + slot_of(xk)));
              if (n + 2 == it.n_tiles) mma_commit(bar(kBarQFree));
            }
          }
          if (!ok) break;
        }
        mma_commit(bar(kBarOFinal));
        if (!ok) break;
        ring += 2 * it.n_tiles;
        t += it.n_tiles;
      }
      if (!ok) {
        // make sure no product is still writing TMEM before it is released
        mma_commit(bar(kBarDrain));
        mbar_wait(bar(kBarDrain), 0, p.err);
      }
    }
    had_item = __shfl_sync(0xffffffffu, had_item ? 1 : 0, 0) != 0;
  } else if (kSplit && warp < 4) {
    had_item = __all_sync(0xffffffffu, wait_for_item(bar(kBarItemFull), 0, s_abort, p.err)) && items[0].n_tiles >= 0;
  } else if (warp == 2) {
    // =========================== rows that are computed again ===========================
    for (int k = 0;; ++k) {
      if (!__all_sync(0xffffffffu, wait_for_item(bar(kBarItemFull + (k & 1)), (k >> 1) & 1, s_abort, p.err))) break;
      if (items[k & 1].n_tiles < 0) break;
      // one barrier to each of two items: the softmax warps cannot be done with item k + 2 before this warp has let go of
      // item k, but with k + 1 they can
      if (!__all_sync(0xffffffffu, wait_or_abort(bar(kBarRows + (k & 1)), (k >> 1) & 1, s_abort, p.err))) break;
      if (__any_sync(0xffffffffu, s_again[(k & 1) * kSoftmaxWarps + (lane & (kSoftmaxWarps - 1))] != 0))
        item_again<E>(p, k & 1);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarItemFree + (k & 1)));
    }
  } else if (warp >= 4) {
    // =========================== softmax groups ===========================
    // Where a thread works follows from its number u among the softmax threads: 256 to a group, of these 128 to a half of
    // a tile's keys, of these 32 to a warp. It is taken apart anew in each part of the item: kept over the loop over the
    // tiles it would cost the registers that the scores need (chunk of 5000 on 7001 with a bias 405 us kept, 338 anew).
    // P and the ranges lie in its order.
    struct Place {
      int u;
      __device__ int lane() const { return u & 31; }
      __device__ int g() const { return u >> 8; }
      __device__ int half() const { return (u >> 7) & 1; }
      __device__ int warp() const { return u >> 5; }
      __device__ int quarter() const { return (u >> 5) & 3; }
      __device__ int row() const { return u & 127; }                // within the group's tile == TMEM lane
      __device__ int barrier() const { return ((u >> 5) & 11) | 4; }  // of the two warps of 32 rows
    };
    auto place = [&]() {
      int t;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
      return Place{t - 128};
    };
    auto tmem_at = [&](const Place& w, int first) {
      return tmem + (static_cast<uint32_t>(w.u & 96) << 16) + first + ((w.u & 384) >> 1);
    };
    auto seen_at = [&](const Place& w) { return sbase + kOffSeen + w.warp() * 16; };
    auto p_row = [&](const Place& w) { return sbase + kOffP + w.u * 128; };
    auto max_for = [&](int u) { return sbase + kOffP + u * 128 + (u & 31) * 4; };
    const float sl2 = p.scale_log2;
    // Named barrier of the two warps of 32 rows. Both come to it equally often whatever happens, so it needs no time
    // limit: they agree on whether to go on before every item, and then come to it once per tile and twice at the end.
    auto pair_sync = [](const Place& w) { asm volatile("bar.sync %0, 64;" ::"r"(w.barrier()) : "memory"); };
    auto pair_agree = [](const Place& w, bool yes) {
      uint32_t all;
      asm volatile(
          "{\n\t.reg .pred q, r;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.and.pred r, %2, 64, q;\n\tselp.u32 %0, 1, 0, r;\n\t}"
          : "=r"(all)
          : "r"(yes ? 1u : 0u), "r"(w.barrier())
          : "memory");
      return all != 0;
    };
    const bool by_maximum = !kCap || kBias || !p.fixed;
    uint32_t parity = 0;  // of the scores' barrier
    bool ok = true;
    for (int k = 0;; ++k) {
      if (ok) ok = __all_sync(0xffffffffu, wait_for_item(bar(kBarItemFull + (k & 1)), (k >> 1) & 1, s_abort, p.err));
      const Place w0 = place();
      ok = pair_agree(w0, ok);
      if (!ok) break;
      const Item& it = items[k & 1];
      if (it.n_tiles < 0) break;
      int pos, lo, hi;
      seen_from(p, it, it.r0 + (p.neighbours && w0.g() > 0 ? kBM : 0) + w0.row(), pos, lo, hi);
      // seen by any and by all of the warp's rows
      {
        const int any_lo = __reduce_min_sync(0xffffffffu, lo < hi ? lo : INT32_MAX);
        const int any_hi = __reduce_max_sync(0xffffffffu, lo < hi ? hi : 0);
        const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
        if (w0.lane() == 0)
          asm volatile("st.shared.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(seen_at(w0)), "r"(any_lo), "r"(any_hi), "r"(all_lo),
                       "r"(all_hi)
                       : "memory");
        __syncwarp();
      }
      const int min_pos = __reduce_min_sync(0xffffffffu, pos);
      const float slope = kBias ? p.slopes[it.head0 + (p.neighbours ? 0 : w0.g())] * kLog2e : 0.f;
      float m = -INFINITY;  // the row's reference, log2 units; within 8 (and kLift) of its running maximum from below, or 0
      float l = 0.f;        // of this thread's keys
      constexpr int kStep = kBack ? -kBN : kBN;
      int key0 = first_key_of(it, 0) + w0.half() * kCols - kStep;
      for (int left = it.n_tiles; left > 0; --left) {
        key0 += kStep;
        const Place w = place();
        int any_lo, any_hi, all_lo, all_hi;
        asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(any_lo), "=r"(any_hi), "=r"(all_lo), "=r"(all_hi)
                     : "r"(seen_at(w))
                     : "memory");
        // every lane waits (each needs the acquire); the warp then agrees, so
        // the warp-collective tensor-memory loads below run on all 32 lanes
        if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(bar(kBarSFull + w.g()), parity, s_abort, p.err));
        if (!ok) {  // the other warp of these rows may still come to the pair's barrier
          if (by_maximum) pair_sync(w);
          continue;
        }
        parity ^= 1;
        tc_fence_after();
        const bool none = key0 + kCols <= any_lo || key0 >= any_hi;  // no row sees any of these keys
        const bool edge = key0 < all_lo || key0 + kCols > all_hi;  // some row does not see all of them
        float s[kCols], mx = -INFINITY;
        const float base = m == -INFINITY ? 0.f : m;
        if (!none) {
          {
            uint32_t x0[32], x1[32];
            const uint32_t tS = tmem_at(w, 0);
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
            if (key0 + kCols > any_hi) {  // what lies behind the rows' keys has no say in how their scores are worked out
#pragma unroll
              for (int j = 0; j < kCols; ++j) s[j] = j < any_hi - key0 ? s[j] : 0.f;
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
          if (edge) {  // some row does not see all of the keys
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
          // The reference moves to the row's largest score (less kLift) when that is above it by more than 8 (2^8 of
          // headroom), and to the first tile's in which the row sees a key. Its two threads tell one another theirs as they are: rounded to
          // 16 bits, a largest score of 8192 could lie 32 below the reference, and all of the row's p below fp16's range.
          // Either writes it into the other's row of P, a word to a lane, which the other reads before it writes P there:
          // the row's last product is complete once the tile's scores are there, and its threads have met since they last
          // used it (for P, or for the item before).
          const Place wm = place();
          float others;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(max_for(wm.u ^ 128)), "f"(mx) : "memory");
          pair_sync(wm);
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(others) : "r"(max_for(wm.u)) : "memory");
          const float to = fmaxf(mx, others) - kLift<E>;
          const bool move = to > (m == -INFINITY ? m : m + 8.f);
          if (__any_sync(0xffffffffu, move)) {
            const float delta = move ? base - to : 0.f;
            const uint64_t less = f32x2_pack(delta, delta);
#pragma unroll
            for (int j = 0; j < kCols; j += 2) f32x2_unpack(f32x2_add(f32x2_pack(s[j], s[j + 1]), less), s[j], s[j + 1]);
            const float alpha = !move ? 1.f : (m == -INFINITY ? 0.f : ex2_approx(m - to));
            const bool rescale = move && m != -INFINITY;
            if (move) m = to;
            l *= alpha;
            if (__any_sync(0xffffffffu, rescale)) {
              // the running output too (PV of the tile before is complete: S of this one was issued after it)
              const uint32_t tO = tmem_at(wm, 256);
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
        // P = 2^s, rounded to the element type, into the swizzled K-major A tile (eight addresses, made here: kept over the
        // loop they would cost the registers that the scores need)
        const Place wp = place();
        const uint32_t to_p = p_row(wp) | (wp.u & 7) << 4;
        if (!none) {
#pragma unroll
          for (int c = 0; c < kCols / 8; ++c) {
#pragma unroll
            for (int j = c * 8; j < c * 8 + 8; ++j) s[j] = ex2_approx(s[j]);
            const float* e = s + c * 8;
            sts128(to_p ^ (c << 4), Ops::pack(e[0], e[1]), Ops::pack(e[2], e[3]), Ops::pack(e[4], e[5]),
                   Ops::pack(e[6], e[7]));
          }
        } else {
#pragma unroll
          for (int c = 0; c < kCols / 8; ++c) sts128(to_p ^ (c << 4), 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (wp.lane() == 0) mbar_arrive(bar(kBarPReady + wp.g()));
        // The row sum is not needed for P: add it up after P is handed over. Where rows may see few keys, of the rounded p,
        // which is what V is multiplied by, so that their shares add up to 1 exactly (a row that sees one key gets its
        // value as it is); in sums over many keys the roundings do not add up (everywhere it would cost 5 to 9 %).
        if (!none) {
          if (edge) {
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
      if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(bar(kBarOFinal), k & 1, s_abort, p.err));
      // Epilogue, with the item's description read again. Every product is complete, so the warp's part of P is free: a
      // row's two threads add up their sums through it.
      const Item* described = items + (k & 1);
      asm volatile("" : "+l"(described)::"memory");
      const int Lq = described->Lq, cq0 = described->cq0;
      const Place w1 = place();
      const int g = w1.g(), half = w1.half(), row = w1.row(), lane = w1.lane();
      const uint32_t prow = p_row(w1), tO = tmem_at(w1, 256);
      const uint32_t other = half ? prow - kHalfBytes : prow + kHalfBytes;
      if (ok) asm volatile("st.shared.f32 [%0], %1;" ::"r"(prow), "f"(l) : "memory");
      pair_sync(w1);
      if (ok) {
        float more;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(more) : "r"(other) : "memory");
        l += more;
      }
      pair_sync(w1);
      if constexpr (kSplit) {
        // The parts' references and sums are exchanged; then every row is scaled for the common ones and goes to the CTA
        // that adds up its parts, in their order: rows_own of the 256 rows each. Q, P and the ring are idle in every CTA
        // by then; the rows arrive where Q and P were.
        const int rows_own = 2 * kBM / parts, ri = g * kBM + row;
        const uint32_t ml = sbase + kOffKV;
        float ref = by_maximum ? m : 0.f;
        if (!ok || described->n_tiles == 0) {
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
        const uint32_t sums = ml + 2 * kBM * 8;  // for this CTA's own rows
        if (half == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(sums + ri * 4), "f"(L) : "memory");
        const uint32_t dst = in_part(sbase + kOffQ + (part * rows_own + ri % rows_own) * 512, ri / rows_own);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t x[32];
          if (ok && described->n_tiles > 0) {
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
        if (lane == 0) mbar_arrive(bar(kBarDone));
        cluster_sync();
        for (int lr = warp - 4; lr < rows_own; lr += kSoftmaxWarps) {
          const int r2 = part * rows_own + lr, g2 = r2 / kBM, q_row = r2 % kBM;
          const int seq_row = it.r0 + q_row + (p.neighbours ? g2 * kBM : 0), to_head = it.head0 + (p.neighbours ? 0 : g2);
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
          float sum;  // NaN where a score is: so is the row, then
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sum) : "r"(sums + r2 * 4) : "memory");
          if (!isnan(sum) && __any_sync(0xffffffffu, isnan(fmaf(o.x, 0.f, fmaf(o.y, 0.f, fmaf(o.z, 0.f, o.w * 0.f)))))) {
            split_row_again<E>(p, it, to_head, seq_row, rows_went_on(s_abort));
          } else {
            *(reinterpret_cast<uint2*>(p.out + (out_row * p.hq + to_head) * kHeadDim) + lane) =
                make_uint2(Ops::pack(o.x, o.y), Ops::pack(o.z, o.w));
          }
        }
        wait_for_others();
        return;
      }
      // The warp stages its 64 dims of its normalised rows there (128 B a row, 16-byte chunks rotated by the row) and stores
      // them, four rows at once. Rows that are to be computed again are left to warp 2.
      const uint32_t to_p = prow | (lane & 7) << 4;
      const int row0 = described->r0 + (p.neighbours && g > 0 ? kBM : 0) + w1.quarter() * 32;  // of the sequence
      uint32_t again = 0;
      if (ok) {
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float spoilt = 0.f;  // NaN once any element is not finite
        // sixteen columns at once: 32 made the compiler spill scores in the loop over the tiles (351 us became 590)
#pragma unroll 1
        for (int c = 0; c < kCols / 8; c += 2) {
          uint32_t r[2][8];
#pragma unroll
          for (int a = 0; a < 2; ++a) tmem_ld8(tO + (c + a) * 8, r[a]);
          tmem_wait_ld();
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            tmem_reg_fence8(r[a]);
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              x[j] = __uint_as_float(r[a][j]);
              spoilt = fmaf(x[j], 0.f, spoilt);
            }
            sts128(to_p ^ ((c + a) << 4), Ops::pack(x[0] * inv, x[1] * inv), Ops::pack(x[2] * inv, x[3] * inv),
                   Ops::pack(x[4] * inv, x[5] * inv), Ops::pack(x[6] * inv, x[7] * inv));
          }
        }
        again = __ballot_sync(0xffffffffu, isnan(spoilt) && !isnan(inv) && row0 + lane < Lq);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarOFree + g));
      if (ok) {
        const uint32_t stage = prow - lane * 128;
        const int64_t step = static_cast<int64_t>(p.hq) * kHeadDim;
        uint16_t* to = p.out + (static_cast<int64_t>(cq0 + row0) * p.hq + described->head0 + (p.neighbours ? 0 : g)) * kHeadDim +
                       half * kCols + (lane & 7) * 8 + (lane >> 3) * step;
#pragma unroll 4
        for (int rr = lane >> 3; rr < 32; rr += 4, to += 4 * step) {
          uint32_t x0, x1, x2, x3;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                       : "r"(stage + rr * 128 + (((lane ^ rr) & 7) << 4))
                       : "memory");
          if (row0 + rr < Lq) *reinterpret_cast<uint4*>(to) = make_uint4(x0, x1, x2, x3);
        }
      }
      __syncwarp();
      if (lane == 0) {
        s_again[(k & 1) * kSoftmaxWarps + w1.warp()] = again;
        mbar_arrive(bar(kBarRows + (k & 1)));
        mbar_arrive(bar(kBarItemFree + (k & 1)));
      }
    }
    // every softmax warp comes here, whatever happened (a split item's leave above): its last tensor-memory read is complete
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarDone));
    if (kSplit) wait_for_others();
    return;
  }

  if (kSplit && had_item) {  // (warps 0 to 3 here) every thread of a cluster comes to both of its barriers
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    // TMEM is released after every softmax warp's last tensor-memory read. The wait is time-bounded but ignores the abort
    // flag: the softmax warps always arrive.
    __syncwarp();
    mbar_wait(bar(kBarDone), 0, p.err);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (kSplit) {
    if (had_item) cluster_sync();
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
