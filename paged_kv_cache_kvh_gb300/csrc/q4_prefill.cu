// q4_prefill.cu -- causal variable-length attention on tcgen05 whose keys and
// values all sit in the 4-bit paged cache.
//
// The operation is that of prefill.cu: query row i of sequence b sits at
// position Lk_b - Lq_b + i and attends to keys 0..that position. A key's element is
// s * c + z (q4.cuh) rounded to the rows' type, as pkv_load_kvcache_q4 returns it,
// since Q K^T takes operands of one type. V and P are free of that, and fp16 holds
// both (|V| <= 65504, P < 2^14) with 3 bits more than bf16: the second product is
// fp16 for either type of rows (bf16 error against 64 bits 0.0030 -> 0.0022, the
// result's own rounding being 0.0017; no difference in time). Maxima, sums and
// accumulators are fp32. What the call saves is reading the rows back first: 512
// bytes written and read again per (token, kv head), for every sequence that
// shares a prefix.
//
// One CTA computes a 128-row query tile of one sequence for two query heads of
// one kv head, so a K or V tile is widened once for two products; where sequences
// have many query tiles, two CTAs take neighbouring ones and widen half of each
// tile for both (Share):
//   warp 0        loads the Q tiles by TMA
//   warp 1        allocates TMEM and issues every tcgen05.mma
//   warps 4-7     softmax of the first head   (thread = TMEM lane = query row)
//   warps 8-11    softmax of the second head
//   warps 12-19   widen K_n, V_n (128 keys x 128 dims) into a ring of 5 tiles
// (warps 2, 3 only make up the warpgroup for the register split.) P is written
// over the logits in TMEM, as 16-bit pairs, and is the A operand of the second
// product from there: the 64 KB of shared memory that two P tiles would take are
// two more K/V tiles.
//
// A widening warp takes 16 keys of a tile: two batches of 8 keys, 16 bytes of
// codes a lane, which are 8 dims of each of the 4 groups. A batch's registers are
// loaded again for the next tile as soon as it is widened, so a tile's loads are
// in flight while the other batch is converted and the ring slot is waited for.
// A pair of bf16 keys costs two ANDs, one packed multiply-add and one conversion
// (the nibbles are used in place, as fp32 subnormals; see dequantise8), which is why
// a bf16 K tile holds 2^-64 of the values; the powers of two are taken out of the
// logits. Rows past the sequence are written as zeros. So is a group of V that
// reads back as NaN: in a product it would reach every query row of the tile,
// masked or not (0 * NaN). The first such position of each group is kept instead,
// and rows at or past it get NaN in the epilogue.
//
// Registers: 640 threads x 96 at launch, split over the warpgroups so that as little
// as possible spills (shared memory leaves no L1 for local memory: the first form,
// which spilled in its loops, took 904 us where this takes 481). What the compiler
// still spills: 20 bytes in the bf16 form whose keys are split, 8 in the fp16 form of
// many short tiles, nothing in the others. Other splits of those two were no better:
// 152 registers for the softmax, as bf16 has, in the latter (36 bytes; 128 prompts on
// a prefix 474 -> 512 us) and in the former (28 bytes; 512 on 16384 85 -> 86 us).
//
// A tile's start is a chain of loads: lengths, block, codes, first widening, first
// product, about 3 us in all beside 0.6 us between two CTAs and 1.8 us of epilogue.
// So the first block is read with the lengths (486 -> 481 us on the first case
// below), and a pair's first codes go out before it is set up, which waits for
// both CTAs (328 -> 320 on the second; in the other forms the loop became slower
// by more than that).
//
// The issuing warp runs its loop as a whole and elects a thread for each product:
// operand addresses then stay in uniform registers, and with TMEM addresses as
// constants an issue is a few instructions. One thread that computed them in its
// own registers cost 4 % (496 -> 480 us): the issue order is the products' order,
// and the warp competes with four busy ones for its scheduler.
//
// What bounds it: the products (the logits' operands come from shared memory at
// its full rate, two 4 KB tiles in 64 cycles), the softmax of one head's tile
// between them, and the widening, all on the same schedulers. A key tile takes
// 2.0-2.4 us, in pairs 1.7: about 4.5 k warp instructions of widening (a pair's
// CTA: half) and 6 k of softmax, against 2048 cycles (1.1 us) of tensor core at its
// peak. 128 prompts of 64..512 tokens on a shared prefix of 1024 (16 query heads on
// 8): 481 us a CTA to a tile (the tensor pipe active 42 % of the time, instructions
// issued in 56 % of the cycles), 427 us, 0.83 PFLOP/s, in units; 5000 tokens after
// 7001, in pairs, replayed from a graph: 321 us, 1.21 PFLOP/s (fp16 315).
// Measured and not kept, on these two, each beside what the kernel then took: two
// issuing warps, one for each head (528 and 427 beside 480 and 376: the products of
// both mix); no maximum of a tile's logits unless their sum is out of range (506
// and 378 beside 496 and 386: P then waits for the sum); 4 widening warps (581 and
// 461 beside 495 and 386; they are late) and 6 (580 and 545 beside 491 and 457: the
// schedulers have uneven loads); P through shared memory (545 and 515 beside 494
// and 458); logits in 64-key halves with two in flight for each head (630 beside
// 491); waits with a suspend hint or a sleep (same).
// TMEM columns, issue order, the lazily moved maximum and the epilogue are as in
// prefill.cu.
#include <cuda.h>

#include <atomic>
#include <climits>
#include <mutex>
#include <type_traits>

#include "q4.cuh"

namespace pkv {

namespace {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kTileBytes = 128 * kHeadDim * 2;  // 32 KB
constexpr int kHalfBytes = kTileBytes / 2;      // 16 KB: 128 rows x 64 dims
constexpr int kKvSlots = 5;
constexpr int kThreads = 640;
constexpr int kWidenWarps = 8;
constexpr int kWidenWarp0 = 12, kSoftmaxWarp0 = 4;

constexpr int kOffQ = 0;                                 // 2 tiles (and O staging in the epilogue)
constexpr int kOffKV = 2 * kTileBytes;                   // kKvSlots tiles
constexpr int kOffBar = kOffKV + kKvSlots * kTileBytes;  // barriers
constexpr int kBarQ = 0;
constexpr int kBarKvFull = 1;                       // +slot, the widening warps
constexpr int kBarKvFree = kBarKvFull + kKvSlots;   // +slot
constexpr int kBarSFull = kBarKvFree + kKvSlots;    // +g
constexpr int kBarPReady = kBarSFull + 2;           // +g, 4 warps
constexpr int kBarOFinal = kBarPReady + 2;
constexpr int kBarDrain = kBarOFinal + 1;
constexpr int kBarStaged = kBarDrain + 1;           // the 8 softmax warps have staged their O rows
constexpr int kNumBars = kBarStaged + 1;
constexpr int kOffMisc = kOffBar + kNumBars * 8;    // tmem address, abort flag, first NaN position of V's 4 groups
constexpr size_t kSmemBytes = kOffMisc + 32 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "shared memory above the 227 KB a CTA can opt into");

struct Q4PrefillParams {
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* block_tables;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  int32_t bt_stride;
  int32_t num_blocks;
  int32_t num_seqs;
  int32_t max_q_tiles;
  int32_t max_seqlen_q;
  int32_t max_seqlen_k;
  int32_t total_q;
  int32_t hq;
  int32_t hkv;
  float scale_log2;
  const int32_t* items;  // optional tile plan: (qt << 16) | b per item; NULL: all pairs
  int32_t num_items;
  int32_t first;         // the launch's first work item (query tiles x pairs of heads)
  int32_t by_twos;       // items in the order of pairs of neighbouring query tiles (no plan then)
  uint16_t* out;
  unsigned int* err;
};

// kCluster: what another CTA of the cluster did before it arrived is seen as well.
template <bool kCluster>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  if (!kCluster) return mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait that also gives up as soon as another role of the CTA has aborted.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                              unsigned int* err) {
  if (try_wait<kCluster>(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (try_wait<kCluster>(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      flag_error(err, PKV_DEVERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
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
// D[tmem] (+)= A * B[smem desc], kind::f16, issued by one elected thread; the whole
// warp calls these, so that operand addresses are computed once for it, in uniform
// registers. A from shared memory, or (ts) from TMEM: row i in lane i, two 16-bit
// elements to a column.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHiSw128)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHiSw128)
      : "memory");
}
// The issuing thread's products so far arrive on the barrier when they are complete.
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// The same, on the barrier at this place in both CTAs of a pair.
__device__ __forceinline__ void commit_elected_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          bar)
      : "memory");
}
__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok) != 0; }
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// The cluster of CTAs that split the keys of one query tile (kSplit).
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

// Copies within the cluster: dst and bar are in another CTA.
__device__ __forceinline__ void bulk_s2s(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void min_cluster(uint32_t addr, int x) {
  asm volatile("{\n\t.reg .s32 old;\n\tatom.shared::cluster.min.s32 old, [%0], %1;\n\t}" ::"r"(addr), "r"(x) : "memory");
}
// A bf16 K is held as 2^-64 of its values (dequantise8).
template <Elem E>
constexpr float kKeyScale = E == Elem::kBF16 ? 18446744073709551616.f : 1.f;
constexpr float kLift = 6.f;

// One key tile of one query row (a thread's): logits from TMEM, P over them, the
// running maximum m (less kLift, log2 units) and sum l. Where `masked`, keys
// j <= lim are visible. kMayMiss: the first tiles may hold none.
template <bool kMayMiss>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, bool first, bool masked, int lim, float sl2,
                                             float& m, float& l, uint32_t p_ready, int lane) {
  float s[128];
  {
    uint32_t r0_[32], r1[32], r2[32], r3[32];
    tmem_ld32(tS + 0, r0_);
    tmem_ld32(tS + 32, r1);
    tmem_ld32(tS + 64, r2);
    tmem_ld32(tS + 96, r3);
    tmem_wait_ld();
    tmem_reg_fence(r0_);
    tmem_reg_fence(r1);
    tmem_reg_fence(r2);
    tmem_reg_fence(r3);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      s[j] = __uint_as_float(r0_[j]);
      s[32 + j] = __uint_as_float(r1[j]);
      s[64 + j] = __uint_as_float(r2[j]);
      s[96 + j] = __uint_as_float(r3[j]);
    }
  }
  if (masked) {
#pragma unroll
    for (int j = 0; j < 128; ++j)
      if (j > lim) s[j] = -INFINITY;
  }
  float ma = s[0], mb = s[1];
#pragma unroll
  for (int j = 2; j < 126; j += 4) {
    ma = fmax3(ma, s[j], s[j + 1]);
    mb = fmax3(mb, s[j + 2], s[j + 3]);
  }
  float mx = fmaxf(fmax3(ma, s[126], s[127]), mb);
  mx *= sl2;
  float m_use = m;
  // Move the maximum only when it grows by more than 2^8. m is kLift below it: P stays
  // under 2^14, and is a normal fp16 number down to 2^-20 of the largest.
  if (mx > m + (8.0f + kLift)) m_use = mx - kLift;
  const float alpha = (m == -INFINITY) ? 0.f : ex2_approx(m - m_use);
  l *= alpha;
  const uint64_t sl2x2 = f32x2_pack(sl2, sl2);
  const float neg_m = kMayMiss && m_use == -INFINITY ? 0.f : -m_use;  // a part may begin with keys that a row can't see
  const uint64_t negm2 = f32x2_pack(neg_m, neg_m);
  // P = 2^(s*sl2 - m_use), rounded to fp16 (for either type of rows), over the logits in TMEM
  uint64_t sums[4] = {0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t pk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = c * 16 + 2 * i;
      float a0, a1;
      f32x2_unpack(f32x2_fma(f32x2_pack(s[j], s[j + 1]), sl2x2, negm2), a0, a1);
      a0 = ex2_approx(a0);
      a1 = ex2_approx(a1);
      sums[i & 3] = f32x2_add(sums[i & 3], f32x2_pack(a0, a1));
      pk[i] = ElemOps<Elem::kF16>::pack(a0, a1);
    }
    tmem_st8(tS + c * 8, pk);
  }
  m = m_use;
  // rescale the running output (PV_g(n-1) is complete: S_g(n) was issued after it)
  if (!first && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
    for (int c = 0; c < 16; ++c) {
      uint32_t r[8];
      tmem_ld8(tO + c * 8, r);
      tmem_wait_ld();
      tmem_reg_fence8(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
      tmem_st8(tO + c * 8, r);
    }
  }
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(p_ready);
  {
    float t0, t1, t2, t3, t4, t5, t6, t7;
    f32x2_unpack(sums[0], t0, t1);
    f32x2_unpack(sums[1], t2, t3);
    f32x2_unpack(sums[2], t4, t5);
    f32x2_unpack(sums[3], t6, t7);
    l += ((t0 + t1) + (t2 + t3)) + ((t4 + t5) + (t6 + t7));
  }
}

// A lane's share of one key: 16 bytes of codes (8 dims of each of the 4 groups) and
// the 4 parameters.
struct KeyShare {
  uint4 codes, par;
};
__device__ __forceinline__ void load_key(const Q4PrefillParams& p, KeyShare& s, bool of_v, int blk, int kv_head, int key0,
                                         int row, int lane, int Lk) {
  s.codes = s.par = make_uint4(0, 0, 0, 0);
  if (blk < 0 || key0 + row >= Lk) return;  // zeros: a scale and a minimum of 0
  const uint8_t* base = (of_v ? p.v_cache : p.k_cache) +
                        (static_cast<int64_t>(blk) * p.hkv + kv_head) * kQ4RecordBytes +
                        (key0 % kBlockSize + row) / kQ4Tile * kQ4TileBytes;
  const int tok = row % kQ4Tile;
  s.codes = __ldg(reinterpret_cast<const uint4*>(base + tok * kQ4CodeBytes + (lane & 3) * 16));
  s.par = __ldg(reinterpret_cast<const uint4*>(base + kQ4TileParams + tok * kQ4ParamBytes));
}
__device__ __forceinline__ int checked_block(const Q4PrefillParams& p, int blk) {
  if (blk >= 0 && blk < p.num_blocks) return blk;
  flag_error(p.err, PKV_DEVERR_BAD_BLOCK);
  return -1;
}
// s -> key `row` of the K or V tile at `tile`; `reload` fills s again meanwhile,
// on_nan(group) is called where a group of V is NaN (it is written as zeros).
template <Elem E, bool kV, class Reload, class OnNan>
__device__ __forceinline__ void widen_key(KeyShare& s, uint32_t tile, int row, int lane, Reload reload, OnNan on_nan) {
  const bool odd = (lane >> 2) & 1;
  uint32_t w[4] = {s.codes.x, s.codes.y, s.codes.z, s.codes.w};
  uint32_t sz[4] = {s.par.x, s.par.y, s.par.z, s.par.w};
  int tt = lane & 3;
  if constexpr (kV) {
    // two 8-byte chunks of V: per group, the 4 dims of the first and then of the second
    const uint4 c = s.codes;
    w[0] = __byte_perm(c.x, c.z, 0x5410);
    w[1] = __byte_perm(c.x, c.z, 0x7632);
    w[2] = __byte_perm(c.y, c.w, 0x5410);
    w[3] = __byte_perm(c.y, c.w, 0x7632);
    tt ^= (row & 4) >> 1;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((sz[k] & 0x7fffu) > 0x7c00u) {  // a NaN scale
        on_nan(k);
        sz[k] = 0u;
      }
  }
  reload();
  // odd rows take the groups in another order, so that the 8 lanes of a
  // store phase (two rows, four chunks each) hit all banks
  const uint32_t wa = odd ? w[1] : w[0], wb = odd ? w[0] : w[1], wc = odd ? w[3] : w[2], wd = odd ? w[2] : w[3];
  const uint32_t pa = odd ? sz[1] : sz[0], pb = odd ? sz[0] : sz[1];
  const uint32_t pc = odd ? sz[3] : sz[2], pd = odd ? sz[2] : sz[3];
  const uint32_t at = tile + row * 128;
  const int ca = (odd ? 4 : 0) + tt, cb = (odd ? 0 : 4) + tt;  // 16-byte chunk within the half row
  auto put = [&](uint32_t codes8, uint32_t param, int half, int chunk) {
    const uint4 v = kV ? dequantise8<Elem::kF16>(codes8, param) : dequantise8<E, true>(codes8, param);
    sts128(at + half * kHalfBytes + ((chunk ^ (row & 7)) << 4), v.x, v.y, v.z, v.w);
  };
  put(wa, pa, 0, ca);
  put(wb, pb, 0, cb);
  put(wc, pc, 1, ca);
  put(wd, pd, 1, cb);
}
// The products of one key tile and head: logits from Q and K tiles (low halves of
// their descriptors), output from P in TMEM and a V tile.
template <Elem E>
__device__ __forceinline__ void issue_logits(int g, uint32_t q_lo, uint32_t k_lo) {
  constexpr uint32_t idesc = idesc_f16kind_f32(kBM, kBN, false, false, ElemOps<E>::kMmaFormat);
#pragma unroll
  for (int ks = 0; ks < kHeadDim / 16; ++ks) {
    const uint32_t off = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
    mma_ss(g * 128, q_lo + g * (kTileBytes >> 4) + off, k_lo + off, idesc, ks > 0 ? 1u : 0u);
  }
}
__device__ __forceinline__ void issue_output(int g, uint32_t v_lo, bool first) {
  constexpr uint32_t idesc = idesc_f16kind_f32(kBM, kHeadDim, false, true, ElemOps<Elem::kF16>::kMmaFormat);
#pragma unroll
  for (int ks = 0; ks < kBN / 16; ++ks)
    mma_ts(256 + g * 128, g * 128 + ks * 8, v_lo + ((ks * 16 * 128) >> 4), idesc, ks > 0 || !first ? 1u : 0u);
}

// kWhole: a CTA has a query tile and all its keys. kSplitKeys: the CTAs of a
// cluster have parts of one tile's keys. kPaired: two CTAs have neighbouring query
// tiles of a sequence. Each widens 64 keys of every tile and copies them to the
// other (1 KB bulk copies between their shared memories, which arrive on the
// other's barriers; stores to the other one directly took 520 us where these take
// 329). A slot is free when both have used it.
enum class Share { kWhole, kSplitKeys, kPaired };

template <Elem E, Share kShare>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_q4_kernel(const __grid_constant__ CUtensorMap tm_q, const Q4PrefillParams p) {
  using Ops = ElemOps<E>;
  constexpr bool kSplit = kShare == Share::kSplitKeys, kPair = kShare == Share::kPaired;
  // Registers per thread: 128 * (sum over the five warpgroups) is what the launch holds.
  constexpr int kRegsFirst = kShare == Share::kWhole ? 64 : 80, kRegsSoftmax = 144;
  constexpr int kRegsWiden = kShare == Share::kWhole ? 64 : 56;
  static_assert(kRegsFirst + 2 * kRegsSoftmax + 2 * kRegsWiden == 5 * 96, "the split must sum up to the launch's registers");
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte alignment for the 128-byte-swizzle atoms.
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_addr);
  const uint32_t bar0 = sbase + kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* s_nan = reinterpret_cast<int*>(smem + kOffMisc + 8);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // ---- work item: (query tile, sequence, pair of query heads), longest tiles first ----
  const int pairs = p.hq / 2;
  const int parts = kSplit ? cluster_parts() : 1, part = kSplit ? cluster_part() : 0;
  const int rank = kPair ? cluster_part() : 0;
  int qt, b, pair;
  {
    const int item = p.first + static_cast<int>(blockIdx.x) / parts;
    const int column = (p.by_twos ? item >> 1 : item) / pairs;
    pair = (p.by_twos ? item >> 1 : item) % pairs;
    if (p.items) {
      const int code = p.items[column];
      qt = code >> 16;
      b = code & 0xffff;
    } else {
      const int level = column / p.num_seqs;
      qt = p.max_q_tiles - 1 - (p.by_twos ? 2 * level + (item & 1) : level);
      b = column % p.num_seqs;
      if (!kPair && qt < 0) return;  // the place beside an odd number of tiles
    }
  }
  if (b >= p.num_seqs || (!kPair && qt < 0)) {  // a plan for other cu_seqlens: skip the item
    if (threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
    return;
  }
  const int cq0 = p.cu_q[b], cq1 = p.cu_q[b + 1], ck0 = p.cu_k[b], ck1 = p.cu_k[b + 1];
  const int first_block = kSplit ? -1 : p.block_tables[static_cast<int64_t>(b) * p.bt_stride];
  if (threadIdx.x == 0) {  // (while the lengths are on their way)
    for (int i = 0; i < kNumBars; ++i) {
      int count = 1;
      if (i >= kBarKvFull && i < kBarKvFull + kKvSlots) count = kWidenWarps;
      if (kPair && i >= kBarKvFree && i < kBarKvFree + kKvSlots) count = 2;
      if (i == kBarPReady || i == kBarPReady + 1) count = 4;
      if (i == kBarStaged) count = 8;
      mbar_init(bar(i), count);
    }
    *s_abort = 0;
    for (int i = 0; i < 4; ++i) s_nan[i] = INT_MAX;
    mbar_fence_init();
    prefetch_tmap(&tm_q);
  }
  const int Lq = cq1 - cq0, Lk = ck1 - ck0;
  if (Lq < 0 || Lk < Lq || Lq > p.max_seqlen_q || Lk > p.max_seqlen_k || Lk > INT_MAX - 2 * kBN || cq0 < 0 || cq1 > p.total_q ||
      Lk > static_cast<int64_t>(p.bt_stride) * kBlockSize) {
    if (threadIdx.x == 0 && qt <= 0 && pair == 0 && part == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
    return;
  }
  const int r0 = qt * kBM;
  // (a pair goes on if either of its tiles has a row: the earlier one may be the place
  // beside an odd number of tiles, qt = -1)
  if (max(0, r0 - (kPair ? rank ^ 1 : 0) * kBM) >= Lq) return;
  const int rows_valid = qt < 0 ? 0 : min(kBM, Lq - r0);
  const int pos0 = Lk - Lq + r0;  // position of the tile's first query row
  // key tiles; a pair goes through those of its later tile, as far as that has rows
  const int n_all = (Lk - Lq + min(Lq, r0 + (kPair && rank == 1 ? 2 : 1) * kBM) - 1) / kBN + 1;
  const int tile0 = n_all * part / parts;                    // this CTA's key tiles: from tile0 on
  const int n_tiles = n_all * (part + 1) / parts - tile0;    // (0 only where the keys are split)

  // ---- widening: what a warp loads ----
  const int kv_head = 2 * pair / (p.hq / p.hkv);
  // key of batch 0 within the tile; batch i: + 8 i
  const int row0 = (kPair ? rank * 64 + (warp - kWidenWarp0) * 8 : (warp - kWidenWarp0) * 16) + (lane >> 2);
  auto block_of = [&](int n) -> int {
    return n < n_tiles ? p.block_tables[static_cast<int64_t>(b) * p.bt_stride + (tile0 + n) * kBN / kBlockSize] : -1;
  };
  KeyShare share[2];
  // key `row` of K_{i/2} (even i) or V_{i/2} (odd i), the ring's items, into registers j
  auto load_row = [&](int i, int row, int j, int blk) {
    load_key(p, share[j], i & 1, blk, kv_head, (tile0 + (i >> 1)) * kBN, row, lane, Lk);
  };
  int blk = -1, blk_next = -1;
  if (kPair && warp >= kWidenWarp0) {
    // a warp has one batch of 8 keys, K's in registers 0, V's in registers 1
    blk = checked_block(p, first_block);
    load_row(0, row0, 0, blk);
    load_row(1, row0, 1, blk);
  }

  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(bar(kBarQ), 2 * kTileBytes);
    for (int g = 0; g < 2; ++g) {
      const uint32_t dst = sbase + kOffQ + g * kTileBytes;
      tma_load_3d(dst, &tm_q, 0, 2 * pair + g, cq0 + r0, bar(kBarQ));
      tma_load_3d(dst + kHalfBytes, &tm_q, 64, 2 * pair + g, cq0 + r0, bar(kBarQ));
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (kPair) cluster_sync();  // the other CTA's barriers are there
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they start at column 0

  if (warp < 4) {
    regs_dec<kRegsFirst>();
    if (warp == 0 && lane == 0) mbar_wait(bar(kBarQ), 0, p.err);  // never leave a copy in flight
    if (warp == 1) {
      // =========================== MMA issuer ===========================
      const uint32_t q_lo = desc_lo(sbase + kOffQ, 16);
      const uint32_t k_lo = desc_lo(sbase + kOffKV, 16), v_lo = desc_lo(sbase + kOffKV, kHalfBytes);
      bool ok = all_ok(wait_or_abort(bar(kBarQ), 0, s_abort, p.err));
      int slot = 0;          // of the ring's next tile: K_0, V_0, K_1, ...
      uint32_t parity = 0;
      auto landed = [&]() -> bool {
        return all_ok(wait_or_abort<kPair>(bar(kBarKvFull + slot), parity, s_abort, p.err));
      };
      auto release = [&](int which) {  // once its products are complete
        if (kPair)
          commit_elected_pair(bar(kBarKvFree + which));
        else
          commit_elected(bar(kBarKvFree + which));
      };
      auto advance = [&]() {
        const bool wrap = slot == kKvSlots - 1;
        slot = wrap ? 0 : slot + 1;
        parity ^= wrap ? 1u : 0u;
      };
      auto issue_s = [&](int g, int at) {
        issue_logits<E>(g, q_lo, k_lo + at * (kTileBytes >> 4));
        commit_elected(bar(kBarSFull + g));
      };
      auto issue_pv = [&](int g, int at, bool first) { issue_output(g, v_lo + at * (kTileBytes >> 4), first); };
      if (ok && n_tiles > 0 && (ok = landed())) {
        tc_fence_after();
        issue_s(0, slot);
        issue_s(1, slot);
        release(slot);
        advance();
      }
      for (int n = 0; ok && n < n_tiles; ++n) {
        if (!(ok = landed())) break;
        if (!(ok = all_ok(wait_or_abort(bar(kBarPReady + 0), n & 1, s_abort, p.err)))) break;
        tc_fence_after();
        const int at_v = slot;
        advance();
        const bool more = n + 1 < n_tiles;
        issue_pv(0, at_v, n == 0);
        if (more) {
          if (!(ok = landed())) break;
          tc_fence_after();
          issue_s(0, slot);
        }
        if (!(ok = all_ok(wait_or_abort(bar(kBarPReady + 1), n & 1, s_abort, p.err)))) break;
        tc_fence_after();
        issue_pv(1, at_v, n == 0);
        release(at_v);
        if (more) {
          issue_s(1, slot);
          release(slot);
          advance();
        }
      }
      commit_elected(bar(kBarOFinal));
      if (!ok) {
        // make sure no product is still writing TMEM before it is released
        commit_elected(bar(kBarDrain));
        mbar_wait(bar(kBarDrain), 0, p.err);
      }
    }
    __syncwarp();
    if (kSplit || kPair) cluster_sync();
    if (warp == 1) {
      // TMEM is released after every softmax warp's last tensor-memory read
      mbar_wait(bar(kBarStaged), 0, p.err);
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
    if (kSplit) cluster_sync();
  } else if (warp >= kWidenWarp0) {
    // =========================== K/V widening ===========================
    regs_dec<kRegsWiden>();
    const uint32_t other = kPair ? in_part(sbase, rank ^ 1) : 0u;  // the pair's other CTA
    auto widen_row = [&](auto of_v, int i, int row, int j, uint32_t slot_off, auto reload) {
      widen_key<E, decltype(of_v)::value>(share[j], sbase + kOffKV + slot_off, row, lane, reload, [&](int k) {
        const int at = (tile0 + (i >> 1)) * kBN + row;
        atomicMin(s_nan + k, at);
        if (kPair) min_cluster(other + kOffMisc + 8 + 4 * k, at);
      });
    };
    // the item's slot, once the products (a pair's: of both CTAs) that used it before are complete
    auto wait_slot = [&](int i) -> bool {
      return i < kKvSlots || all_ok(wait_or_abort<kPair>(bar(kBarKvFree + i % kKvSlots), ((i / kKvSlots) - 1) & 1,
                                                         s_abort, p.err));
    };
    auto written = [&](int i) {
      const uint32_t full = bar(kBarKvFull + i % kKvSlots);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (kPair) {
          // the warp's 8 rows to the other CTA, which sends as many
          mbar_arrive_expect_tx(full, 2048);
          const uint32_t rows = sbase + kOffKV + i % kKvSlots * kTileBytes + row0 * 128;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t src = rows + half * kHalfBytes;
            bulk_s2s(src - sbase + other, src, 1024, full - sbase + other);
          }
        } else {
          mbar_arrive(full);
        }
      }
    };
    const int n_items = 2 * n_tiles;
    if constexpr (kPair) {
      for (int i = 0; i < n_items; i += 2) {
        blk_next = block_of((i >> 1) + 1);
        if (!wait_slot(i)) break;
        if (i + 2 < n_items) blk = checked_block(p, blk_next);
        widen_row(std::false_type{}, i, row0, 0, i % kKvSlots * kTileBytes,
                  [&] { if (i + 2 < n_items) load_row(i + 2, row0, 0, blk); });
        written(i);
        if (!wait_slot(i + 1)) break;
        widen_row(std::true_type{}, i + 1, row0, 1, (i + 1) % kKvSlots * kTileBytes,
                  [&] { if (i + 2 < n_items) load_row(i + 3, row0, 1, blk); });
        written(i + 1);
      }
      // the other CTA's last arrivals on this one's barriers
      for (int i = max(0, n_items - kKvSlots); i < n_items; ++i)
        if (!wait_slot(i + kKvSlots)) break;
    } else {
      blk = n_tiles > 0 ? checked_block(p, kSplit ? block_of(0) : first_block) : -1;
#pragma unroll
      for (int j = 0; j < 2; ++j) load_row(0, row0 + 8 * j, j, blk);
      for (int i = 0; i < n_items; i += 2) {
        blk_next = block_of((i >> 1) + 1);
        if (!wait_slot(i)) break;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          widen_row(std::false_type{}, i, row0 + 8 * j, j, i % kKvSlots * kTileBytes,
                    [&] { load_row(i + 1, row0 + 8 * j, j, blk); });
        written(i);
        if (i + 2 < n_items) blk = checked_block(p, blk_next);
        if (!wait_slot(i + 1)) break;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          widen_row(std::true_type{}, i + 1, row0 + 8 * j, j, (i + 1) % kKvSlots * kTileBytes,
                    [&] { if (i + 2 < n_items) load_row(i + 2, row0 + 8 * j, j, blk); });
        written(i + 1);
      }
    }
    __syncwarp();
    if (kSplit || kPair) cluster_sync();  // (a pair: nothing is on its way to this CTA or from it any more)
    if (kSplit) cluster_sync();
  } else {
    // =========================== softmax groups ===========================
    regs_inc<kRegsSoftmax>();
    const int g = (warp - kSoftmaxWarp0) >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;  // query row within the tile == TMEM lane
    const int pos = pos0 + row;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_base + g * 128;
    const uint32_t tO = tmem + lane_base + 256 + g * 128;
    const float sl2 = p.scale_log2 * kKeyScale<E>;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int n = 0; n < n_tiles; ++n) {
      ok = wait_or_abort(bar(kBarSFull + g), n & 1, s_abort, p.err);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int key0 = (tile0 + n) * kBN;
      softmax_tile<kSplit>(tS, tO, n == 0, key0 + kBN - 1 > pos0 || key0 + kBN > Lk, min(pos, Lk - 1) - key0, sl2, m, l,
                           bar(kBarPReady + g), lane);
    }
    if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(bar(kBarOFinal), 0, s_abort, p.err));
    const uint32_t stage = sbase + kOffQ;
    if constexpr (kSplit) {
      // Epilogue of a CTA that had some of the keys. The rows' maxima and sums are
      // exchanged; then every row is scaled for the common maximum and sum and goes
      // to the CTA that adds up its parts, in their order: rows_own of the 256 rows
      // (both heads') each. The ring is idle in every CTA by then.
      const int rows_own = 256 / parts;
      const int ri = g * 128 + row;
      const uint32_t ml = sbase + kOffKV + 4 * kTileBytes;  // behind the 128 KB that rows arrive in
      if (!ok) {
        m = -INFINITY;
        l = 0.f;
      }
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ml + ri * 8), "f"(m), "f"(l) : "memory");
      cluster_sync();
      float M = -INFINITY, L = 0.f;
      for (int i = 0; i < parts; ++i) M = fmaxf(M, ld_cluster_f2(in_part(ml + ri * 8, i)).x);
      if (M == -INFINITY) M = 0.f;
      for (int i = 0; i < parts; ++i) {
        const float2 v = ld_cluster_f2(in_part(ml + ri * 8, i));
        L = fmaf(ex2_approx(v.x - M), v.y, L);
      }
      const float inv = ex2_approx(m - M) * ((L > 0.f ? 1.f / L : L == L ? 0.f : L));
      const uint32_t dst = in_part(stage + (part * rows_own + ri % rows_own) * 512, ri / rows_own);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) {  // group c of 32 dims
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
        for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * inv);
        if (pos >= s_nan[c]) {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0x7fffffffu;
        }
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          st_cluster_f4(dst + (((c * 8 + j / 4) ^ (row & 31)) << 4), __uint_as_float(x[j]), __uint_as_float(x[j + 1]),
                        __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarStaged));
      cluster_sync();
      for (int lr = warp - kSoftmaxWarp0; lr < rows_own; lr += 8) {
        const int r2 = part * rows_own + lr, q_row = r2 & 127;
        if (q_row >= rows_valid) continue;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < parts; ++i) {
          float4 v;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                       : "r"(stage + (i * rows_own + lr) * 512 + ((lane ^ (q_row & 31)) << 4))
                       : "memory");
          o.x += v.x;
          o.y += v.y;
          o.z += v.z;
          o.w += v.w;
        }
        uint2 w;
        w.x = Ops::pack(o.x, o.y);
        w.y = Ops::pack(o.z, o.w);
        *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(cq0 + r0 + q_row) * p.hq + 2 * pair + (r2 >> 7)) * kHeadDim +
                                  lane * 4) = w;
      }
      return;
    }
    if (kPair) cluster_sync();  // NaN positions of both CTAs' keys are known
    // Epilogue: every product is complete, so O is staged in the two Q tiles (both
    // heads of a query row side by side, 512 B, 16-byte chunks rotated by the row)
    // and leaves as whole rows.
    if (ok) {
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
#pragma unroll
      for (int c = 0; c < 4; ++c) {  // group c of 32 dims
        uint32_t r[32];
        tmem_ld32(tO + c * 32, r);
        tmem_wait_ld();
        tmem_reg_fence(r);
        if (pos >= s_nan[c]) {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0x7fffffffu;
        }
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          const int q = g * 16 + c * 4 + j / 8;  // 16-byte chunk of the 512-byte row
          sts128(stage + row * 512 + ((q ^ (row & 31)) << 4),
                 Ops::pack(__uint_as_float(r[j + 0]) * inv, __uint_as_float(r[j + 1]) * inv),
                 Ops::pack(__uint_as_float(r[j + 2]) * inv, __uint_as_float(r[j + 3]) * inv),
                 Ops::pack(__uint_as_float(r[j + 4]) * inv, __uint_as_float(r[j + 5]) * inv),
                 Ops::pack(__uint_as_float(r[j + 6]) * inv, __uint_as_float(r[j + 7]) * inv));
        }
      }
    }
    // all 8 softmax warps arrive, whatever happened, so the waits on it always end
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarStaged));
    const bool staged = __all_sync(0xffffffffu, wait_or_abort(bar(kBarStaged), 0, s_abort, p.err));
    if (ok && staged) {
      uint16_t* obase = p.out + (static_cast<int64_t>(cq0 + r0) * p.hq + 2 * pair) * kHeadDim + lane * 8;
      for (int rr = warp - kSoftmaxWarp0; rr < rows_valid; rr += 8) {
        uint32_t a, b2, c2, d;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a), "=r"(b2), "=r"(c2), "=r"(d)
                     : "r"(stage + rr * 512 + ((lane ^ (rr & 31)) << 4)));
        *reinterpret_cast<uint4*>(obase + static_cast<int64_t>(rr) * p.hq * kHeadDim) = make_uint4(a, b2, c2, d);
      }
    }
  }
}

// ---- the same for many short tiles: every CTA goes through several units ----
//
// One CTA to a tile spends about 5.4 us on each beside its key tiles: 3 us until the
// first logits, 1.8 of epilogue, 0.6 between two CTAs. Here one CTA per SM goes
// through units (a query tile and two heads) k * SMs + its index of a list, a plan's
// or else longest tiles first, that every CTA builds from the lengths, and the roles
// run on from one unit to the next:
//   warp 0       describes the units (kDescs of them are under way at most) and
//                loads a unit's queries as soon as the last one's logits are done
//   warps 12-19  widen the next unit's first tiles while the last products run
//   warp 1       issues the next unit's logits while the softmax warps still write
//                the last output; its first product with V waits until they have
//                read the accumulators
// Outputs leave from registers, 32 bytes a store (the staging area is the queries').
// 128 prompts of 64..512 tokens on a shared prefix of 1024: 480 -> 427 us; 64 of 384
// on 1024 308 -> 290, 16 of 512..1024 on 2048 281 -> 275.
constexpr int kMaxListSeqs = 256, kMaxList = 700, kMaxLevels = 32;  // sequences, tiles, tiles of a sequence
constexpr int kDescs = 4;  // units under way between the loader and the last epilogue
struct UnitInfo {
  int n_tiles;  // < 0: no more
  int b, pair, r0, rows_valid, pos0, Lk, cq0;
};
struct UnitsShared {
  uint64_t bars[32];
  UnitInfo unit[kDescs];
  int nan[kDescs][4];
  uint32_t tmem;
  int abort_flag;
  int list_len;
  uint16_t list[kMaxList];
};
constexpr int kUBarQ = 0, kUBarKvFull = 1, kUBarKvFree = kUBarKvFull + kKvSlots, kUBarSFull = kUBarKvFree + kKvSlots,
              kUBarPReady = kUBarSFull + 2, kUBarOFinal = kUBarPReady + 2, kUBarOFree = kUBarOFinal + 1,
              kUBarQFree = kUBarOFree + 2, kUBarReady = kUBarQFree + 1, kUBarDone = kUBarReady + kDescs,
              kUBarDrain = kUBarDone + kDescs, kUBarEnd = kUBarDrain + 1, kUNumBars = kUBarEnd + 1;
static_assert(kUNumBars <= 32, "barriers");
constexpr size_t kUnitsSmemBytes = kOffBar + sizeof(UnitsShared) + 1024;
static_assert(kUnitsSmemBytes <= 227 * 1024, "shared memory above the 227 KB a CTA can opt into");

// kPlan: the list is a plan's (a form of its own: with both in one, calls without a
// plan took 429 us where they take 424).
template <Elem E, bool kPlan>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_q4_units_kernel(const __grid_constant__ CUtensorMap tm_q, const Q4PrefillParams p) {
  using Ops = ElemOps<E>;
  constexpr int kRegsFirst = 64, kRegsSoftmax = E == Elem::kBF16 ? 152 : 144, kRegsWiden = E == Elem::kBF16 ? 56 : 64;
  static_assert(kRegsFirst + 2 * kRegsSoftmax + 2 * kRegsWiden == 5 * 96, "the split must sum up to the launch's registers");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  UnitsShared* sh = reinterpret_cast<UnitsShared*>(smem_raw + (sbase - raw_addr) + kOffBar);
  const uint32_t bar0 = sbase + kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  volatile int* s_abort = &sh->abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int pairs = p.hq / 2;

  if (threadIdx.x == 32) {
    for (int i = 0; i < kUNumBars; ++i) {
      int count = 1;
      if (i >= kUBarKvFull && i < kUBarKvFull + kKvSlots) count = kWidenWarps;
      if (i >= kUBarPReady && i < kUBarPReady + 2) count = 4;
      if (i >= kUBarOFree && i < kUBarOFree + 2) count = 4;
      if (i >= kUBarDone && i < kUBarDone + kDescs) count = 8;
      if (i == kUBarEnd) count = 8;
      mbar_init(bar(i), count);
    }
    sh->abort_flag = 0;
    mbar_fence_init();
    prefetch_tmap(&tm_q);
  }
  if (warp == 0) {
    // the live query tiles, longest sequences' last ones first (every CTA builds the same list)
    int tiles[kMaxListSeqs / 32];
#pragma unroll
    for (int i = 0; i < kMaxListSeqs / 32; ++i) {
      const int b = i * 32 + lane;
      tiles[i] = 0;
      if (b < p.num_seqs) {
        const int cq0 = p.cu_q[b], cq1 = p.cu_q[b + 1], Lq = cq1 - cq0, Lk = p.cu_k[b + 1] - p.cu_k[b];
        if (Lq < 0 || Lk < Lq || Lq > p.max_seqlen_q || Lk > p.max_seqlen_k || Lk > INT_MAX - 2 * kBN || cq0 < 0 ||
            cq1 > p.total_q || Lk > static_cast<int64_t>(p.bt_stride) * kBlockSize) {
          if (blockIdx.x == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
        } else {
          tiles[i] = (Lq + kBM - 1) / kBM;
        }
      }
    }
    int n = 0;
    if constexpr (kPlan) {
      // a plan's tiles, in its order; what it names beyond a sequence's end is left out
      uint8_t* tiles_of = smem_raw + (sbase - raw_addr) + kOffKV;  // (the ring is not in use yet)
#pragma unroll
      for (int i = 0; i < kMaxListSeqs / 32; ++i) tiles_of[i * 32 + lane] = static_cast<uint8_t>(tiles[i]);
      __syncwarp();
      constexpr int kAhead = 8;
      for (int i0 = 0; i0 < p.num_items; i0 += 32 * kAhead) {
        int code[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) code[k] = p.items[min(i0 + 32 * k + lane, p.num_items - 1)];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int qt = code[k] >> 16, b = code[k] & 0xffff;
          const bool strange = qt < 0 || b >= p.num_seqs;  // a plan for other cu_seqlens
          if (strange && blockIdx.x == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
          const bool take = i0 + 32 * k + lane < p.num_items && !strange && qt < tiles_of[b];
          const uint32_t live = __ballot_sync(0xffffffffu, take);
          if (take) sh->list[n + __popc(live & ((1u << lane) - 1u))] = static_cast<uint16_t>(qt * kMaxListSeqs + b);
          n += __popc(live);
        }
      }
    }
    for (int qt = kPlan ? -1 : p.max_q_tiles - 1; qt >= 0; --qt) {
#pragma unroll
      for (int i = 0; i < kMaxListSeqs / 32; ++i) {
        const uint32_t live = __ballot_sync(0xffffffffu, tiles[i] > qt);
        const int at = n + __popc(live & ((1u << lane) - 1u));
        if (tiles[i] > qt && at < kMaxList) sh->list[at] = static_cast<uint16_t>(qt * kMaxListSeqs + i * 32 + lane);
        n += __popc(live);
      }
    }
    if (lane == 0) {
      if (n > kMaxList && blockIdx.x == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);  // rows given to several sequences
      sh->list_len = min(n, kMaxList);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's, so they start at column 0
  auto ready = [&](int j) -> bool {
    return all_ok(wait_or_abort(bar(kUBarReady + (j % kDescs)), (j / kDescs) & 1, s_abort, p.err));
  };

  if (warp < 4) {
    regs_dec<kRegsFirst>();
    if (warp == 0 && lane == 0) {
      // =========================== units and their queries ===========================
      const int n_units = sh->list_len * pairs;
      int loads = 0;
      for (int j = 0;; ++j) {
        const int d = j % kDescs;
        if (j >= kDescs && !wait_or_abort(bar(kUBarDone + d), ((j / kDescs) - 1) & 1, s_abort, p.err)) break;
        const int64_t unit = static_cast<int64_t>(j) * gridDim.x + blockIdx.x;
        UnitInfo u{};
        u.n_tiles = -1;
        if (unit < n_units) {
          const int code = sh->list[static_cast<int>(unit) / pairs];
          u.b = code % kMaxListSeqs;
          u.pair = static_cast<int>(unit) % pairs;
          u.r0 = code / kMaxListSeqs * kBM;
          u.cq0 = p.cu_q[u.b];
          const int Lq = p.cu_q[u.b + 1] - u.cq0;
          u.Lk = p.cu_k[u.b + 1] - p.cu_k[u.b];
          u.rows_valid = min(kBM, Lq - u.r0);
          u.pos0 = u.Lk - Lq + u.r0;
          u.n_tiles = (u.pos0 + u.rows_valid - 1) / kBN + 1;
        }
        sh->unit[d] = u;
        for (int i = 0; i < 4; ++i) sh->nan[d][i] = INT_MAX;
        mbar_arrive(bar(kUBarReady + d));
        if (u.n_tiles < 0) break;
        if (j > 0 && !wait_or_abort(bar(kUBarQFree), (j - 1) & 1, s_abort, p.err)) break;
        mbar_arrive_expect_tx(bar(kUBarQ), 2 * kTileBytes);
        for (int g = 0; g < 2; ++g) {
          const uint32_t dst = sbase + kOffQ + g * kTileBytes;
          tma_load_3d(dst, &tm_q, 0, 2 * u.pair + g, u.cq0 + u.r0, bar(kUBarQ));
          tma_load_3d(dst + kHalfBytes, &tm_q, 64, 2 * u.pair + g, u.cq0 + u.r0, bar(kUBarQ));
        }
        ++loads;
      }
      if (loads > 0) mbar_wait(bar(kUBarQ), (loads - 1) & 1, p.err);  // never leave a copy in flight
    }
    if (warp == 1) {
      // =========================== MMA issuer ===========================
      const uint32_t q_lo = desc_lo(sbase + kOffQ, 16);
      const uint32_t k_lo = desc_lo(sbase + kOffKV, 16), v_lo = desc_lo(sbase + kOffKV, kHalfBytes);
      bool ok = true;
      int slot = 0;
      uint32_t parity = 0, tile_parity = 0;
      auto landed = [&]() -> bool { return all_ok(wait_or_abort(bar(kUBarKvFull + slot), parity, s_abort, p.err)); };
      auto release = [&](int which) { commit_elected(bar(kUBarKvFree + which)); };
      auto advance = [&]() {
        const bool wrap = slot == kKvSlots - 1;
        slot = wrap ? 0 : slot + 1;
        parity ^= wrap ? 1u : 0u;
      };
      auto issue_s = [&](int g, int at) {
        issue_logits<E>(g, q_lo, k_lo + at * (kTileBytes >> 4));
        commit_elected(bar(kUBarSFull + g));
      };
      auto issue_pv = [&](int g, int at, bool first) { issue_output(g, v_lo + at * (kTileBytes >> 4), first); };
      for (int j = 0; ok; ++j) {
        if (!(ok = ready(j))) break;
        const int n_tiles = sh->unit[j % kDescs].n_tiles;
        if (n_tiles < 0) break;
        if (!(ok = all_ok(wait_or_abort(bar(kUBarQ), j & 1, s_abort, p.err)) && landed())) break;
        tc_fence_after();
        issue_s(0, slot);
        issue_s(1, slot);
        release(slot);
        if (n_tiles == 1) commit_elected(bar(kUBarQFree));
        advance();
        for (int n = 0; n < n_tiles; ++n) {
          const bool more = n + 1 < n_tiles;
          if (!(ok = landed())) break;
          if (!(ok = all_ok(wait_or_abort(bar(kUBarPReady + 0), tile_parity, s_abort, p.err)))) break;
          if (n == 0 && j > 0 && !(ok = all_ok(wait_or_abort(bar(kUBarOFree + 0), (j - 1) & 1, s_abort, p.err)))) break;
          tc_fence_after();
          const int at_v = slot;
          advance();
          issue_pv(0, at_v, n == 0);
          if (more) {
            if (!(ok = landed())) break;
            tc_fence_after();
            issue_s(0, slot);
          }
          if (!(ok = all_ok(wait_or_abort(bar(kUBarPReady + 1), tile_parity, s_abort, p.err)))) break;
          if (n == 0 && j > 0 && !(ok = all_ok(wait_or_abort(bar(kUBarOFree + 1), (j - 1) & 1, s_abort, p.err)))) break;
          tc_fence_after();
          issue_pv(1, at_v, n == 0);
          release(at_v);
          if (more) {
            issue_s(1, slot);
            release(slot);
            if (n + 2 == n_tiles) commit_elected(bar(kUBarQFree));
            advance();
          }
          tile_parity ^= 1;
        }
        commit_elected(bar(kUBarOFinal));
      }
      if (!ok) {
        // make sure no product is still writing TMEM before it is released
        commit_elected(bar(kUBarDrain));
        mbar_wait(bar(kUBarDrain), 0, p.err);
      }
      __syncwarp();
      mbar_wait(bar(kUBarEnd), 0, p.err);
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  } else if (warp >= kWidenWarp0) {
    // =========================== K/V widening ===========================
    regs_dec<kRegsWiden>();
    const int row0 = (warp - kWidenWarp0) * 16 + (lane >> 2);
    int slot = 0;
    uint32_t parity = 1;  // of the slot's last use: nothing to wait for in the first round
    bool ok = true;
    for (int j = 0; ok; ++j) {
      if (!(ok = ready(j))) break;
      const UnitInfo& u = sh->unit[j % kDescs];
      const int n_tiles = u.n_tiles;
      if (n_tiles < 0) break;
      const int Lk = u.Lk;
      const int64_t table = static_cast<int64_t>(u.b) * p.bt_stride;
      const int kv_head = 2 * u.pair / (p.hq / p.hkv);
      int* s_nan = sh->nan[j % kDescs];
      auto block_of = [&](int n) -> int { return n < n_tiles ? p.block_tables[table + n * kBN / kBlockSize] : -1; };
      KeyShare share[2];
      auto load_row = [&](int i, int row, int jj, int blk) {
        load_key(p, share[jj], i & 1, blk, kv_head, (i >> 1) * kBN, row, lane, Lk);
      };
      auto widen_row = [&](auto of_v, int i, int row, int jj, auto reload) {
        widen_key<E, decltype(of_v)::value>(share[jj], sbase + kOffKV + slot * kTileBytes, row, lane, reload,
                                            [&](int k) { atomicMin(s_nan + k, (i >> 1) * kBN + row); });
      };
      auto wait_slot = [&]() -> bool {
        return all_ok(wait_or_abort(bar(kUBarKvFree + slot), parity, s_abort, p.err));
      };
      auto written = [&]() {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kUBarKvFull + slot));
        const bool wrap = slot == kKvSlots - 1;
        slot = wrap ? 0 : slot + 1;
        parity ^= wrap ? 1u : 0u;
      };
      const int n_items = 2 * n_tiles;
      int blk = checked_block(p, block_of(0)), blk_next = -1;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) load_row(0, row0 + 8 * jj, jj, blk);
      for (int i = 0; i < n_items; i += 2) {
        blk_next = block_of((i >> 1) + 1);
        if (!(ok = wait_slot())) break;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
          widen_row(std::false_type{}, i, row0 + 8 * jj, jj, [&] { load_row(i + 1, row0 + 8 * jj, jj, blk); });
        written();
        if (i + 2 < n_items) blk = checked_block(p, blk_next);
        if (!(ok = wait_slot())) break;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
          widen_row(std::true_type{}, i + 1, row0 + 8 * jj, jj,
                    [&] { if (i + 2 < n_items) load_row(i + 2, row0 + 8 * jj, jj, blk); });
        written();
      }
    }
  } else {
    // =========================== softmax groups ===========================
    regs_inc<kRegsSoftmax>();
    const int g = (warp - kSoftmaxWarp0) >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_base + g * 128;
    const uint32_t tO = tmem + lane_base + 256 + g * 128;
    const float sl2 = p.scale_log2 * kKeyScale<E>;
    uint32_t tile_parity = 0;
    bool ok = true;
    for (int j = 0; ok; ++j) {
      if (!(ok = ready(j))) break;
      const UnitInfo& u = sh->unit[j % kDescs];
      const int n_tiles = u.n_tiles, pos0 = u.pos0, Lk = u.Lk;
      if (n_tiles < 0) break;
      const int pos = pos0 + row;
      float m = -INFINITY, l = 0.f;
      for (int n = 0; n < n_tiles; ++n) {
        if (!(ok = all_ok(wait_or_abort(bar(kUBarSFull + g), tile_parity, s_abort, p.err)))) break;
        tile_parity ^= 1;
        tc_fence_after();
        const int key0 = n * kBN;
        softmax_tile<false>(tS, tO, n == 0, key0 + kBN - 1 > pos0 || key0 + kBN > Lk, min(pos, Lk - 1) - key0, sl2, m, l,
                            bar(kUBarPReady + g), lane);
      }
      if (ok) ok = all_ok(wait_or_abort(bar(kUBarOFinal), j & 1, s_abort, p.err));
      if (!ok) break;
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
      const bool valid = row < u.rows_valid;
      uint16_t* orow = p.out + (static_cast<int64_t>(u.cq0 + u.r0 + row) * p.hq + 2 * u.pair + g) * kHeadDim;
      const int* s_nan = sh->nan[j % kDescs];
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {  // group c of 32 dims
        uint32_t r[32];
        tmem_ld32(tO + c * 32, r);
        tmem_wait_ld();
        tmem_reg_fence(r);
        if (c == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kUBarOFree + g));
        }
        if (pos >= s_nan[c]) {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0x7fffffffu;
        }
        uint32_t x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          x[i] = Ops::pack(__uint_as_float(r[2 * i]) * inv, __uint_as_float(r[2 * i + 1]) * inv);
        if (valid) {
#pragma unroll
          for (int i = 0; i < 16; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(orow + c * 32 + 2 * i), "r"(x[i]),
                         "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]),
                         "r"(x[i + 7])
                         : "memory");
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kUBarDone + j % kDescs));
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kUBarEnd));
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static std::atomic<EncodeTiledFn> known;
  EncodeTiledFn fn = known.load(std::memory_order_acquire);
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      known.store(fn = reinterpret_cast<EncodeTiledFn>(ptr), std::memory_order_release);
  }
  return fn;
}

// [rows, heads, 128] view of q, rows row_stride elements apart; box = 128 rows x 1 head x 64 dims.
bool encode_q(CUtensorMap* tm, const void* base, int64_t rows, int heads, int64_t row_stride, Elem elem) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim * 2), static_cast<cuuint64_t>(row_stride * 2)};
  const cuuint32_t box[3] = {64, 1, 128};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = elem == Elem::kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(tm, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kPairTiles = 4, kPairKeyTiles = 28;  // query tiles per sequence, and key tiles, from which on CTAs pair up
constexpr int kUnitRounds = 4;  // rounds of items from which on a CTA goes through several
constexpr int kMinPartTiles = 2;  // key tiles per CTA at least, where the keys of an item are split

template <Elem E, Share kShare>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(prefill_q4_kernel<E, kShare>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kSmemBytes));
}

struct DeviceLimits {
  bool known;
  int sms;
  int clusters[4];  // [i], i > 0: clusters of 2^i CTAs that run at once
};

cudaLaunchConfig_t launch_config(unsigned ctas, int parts, cudaLaunchAttribute* attr, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = static_cast<unsigned>(parts);
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 1 : 0;
  return cfg;
}

template <Elem E>
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
  if ((e = allow_smem<E, Share::kWhole>()) != cudaSuccess || (e = allow_smem<E, Share::kSplitKeys>()) != cudaSuccess ||
      (e = allow_smem<E, Share::kPaired>()) != cudaSuccess ||
      (e = cudaFuncSetAttribute(prefill_q4_units_kernel<E, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kUnitsSmemBytes))) != cudaSuccess ||
      (e = cudaFuncSetAttribute(prefill_q4_units_kernel<E, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kUnitsSmemBytes))) != cudaSuccess)
    return e;
  if ((e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  for (int i = 1; i < 4; ++i) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = launch_config(static_cast<unsigned>(d.sms) << i, 1 << i, &attr, nullptr);
    e = cudaOccupancyMaxActiveClusters(&d.clusters[i], prefill_q4_kernel<E, Share::kSplitKeys>, &cfg);
    if (e != cudaSuccess) return e;
  }
  d.known = true;
  if (dev >= 0 && dev < 64) all[dev] = d;
  *out = d;
  return cudaSuccess;
}

// The items run longest first, one CTA to an SM. What is left of them after whole
// rounds would keep a few SMs busy for one more item, and a call of few items uses
// few SMs from the start. Where all of that rest can run at once with each item's
// keys split over a cluster of 2, 4 or 8 CTAs, it does, as a launch of its own,
// the most parts first that leave a part kMinPartTiles key tiles. Times in key
// tiles (about 2.1 us each): the rest takes `tiles` as it is, less what it fits
// into the first round's uneven end (after an even number of rounds the long and
// the short items have evened out), and tiles / parts when split, plus 2 for the
// merge and 6 for the launch after others.
//   16 query heads on 8   whole  2 parts  4 parts  8 parts   (us, when this was chosen)
//      16 tokens after 512   20.6    21.6     21.3     19.6   kept whole
//     128 after 2048         45.2    34.9     28.8     24.7   8 parts
//     512 after 1024         37.0    28.8     25.7     (59)   4: 32 clusters of 8 don't fit at once
//    1024 after 4096         94.4    59.5      (73)    (128)  2
//    2800 after 1024         74.9    99.5     95.4    112.5   whole: the rest fits into the uneven end
//    3000 after 5000        208.0   203.9    218.2    226.5   whole
//    5000 after 2000        215.2   207.7    200.8    216.2   4
//    5000 after 7001        459.9   412.8    386.2    398.5   4
//
// kUnitRounds rounds of items and more go to the kernel that takes them in units, if
// its list holds them (its stores need 32-byte aligned rows): 29 of 100..1024 94 ->
// 83 us, 200 of 64 on 300 135 -> 108, 40 of 1..400 on 500 96 -> 87; on fewer rounds
// its fixed shares are uneven (4 of 2048 83 -> 97). Without a plan the items are all
// places up to the longest sequence, empty ones among them, of which each costs the
// other forms a CTA: one of 4096 beside 20 of 10 120 -> 112 us (of 1 on 2000: 178 ->
// 145), one of 1024 beside 255 of 1, all on 1000, 433 -> 304. Full rounds behind long
// keys gain nothing (48 of 400 on 2000 494 in either form, 200 of 100 on 2000 470 ->
// 477) or lose (64 of 200 on 4096 549 -> 578, 100 of 300 on 4096 1269 -> 1322); what
// is left over after them, if its keys are split, keeps them from units (128 of 300 on
// 4096 1644, in units 1695).
//
// Pairs of CTAs widen half as much each, 15 % of the time on long keys: one prompt
// of 8192 259 -> 224 us, 16 of 1024 on 4096 589 -> 507, 5000 on 7001 382 -> 329.
// On short ones setting two CTAs up together costs more (8 of 1024 on 1024 124 ->
// 125, 16 of 1024 109 -> 126), and an odd number of tiles leaves one CTA idle
// (32 of 300 on 8192 790 -> 862, 16 of 512..1024 on 2048 286 -> 302): so only where
// sequences have kPairTiles query tiles on average and kPairKeyTiles key tiles. A
// plan's items are not paired (5000 on 7001 321 us without a plan, 356 with one), but it
// leaves out the empty places (one of 4096 beside 20 of 10 112 -> 77 us, one of 8192
// beside 31 of 1 on 2000 437 -> 312).
template <Elem E>
cudaError_t launch_typed(const CUtensorMap& tq, Q4PrefillParams& p, int64_t n_items, int32_t prefix_tiles,
                         cudaStream_t stream) {
  DeviceLimits d;
  cudaError_t e = device_limits<E>(&d);
  if (e != cudaSuccess) return e;
  // pairs: where sequences have query tiles enough that few are left single, and keys enough
  const int64_t columns = p.items ? 1 : static_cast<int64_t>(p.num_seqs) * (p.hq / 2);
  const bool paired = !p.items && p.total_q >= int64_t{kPairTiles} * kBM * p.num_seqs &&
                      prefix_tiles + p.max_q_tiles >= kPairKeyTiles;
  if (paired) n_items = (p.max_q_tiles + 1) / 2 * 2 * columns;
  const int64_t rest = n_items % d.sms, rounds = n_items / d.sms;
  int shift = 0;
  if (rest > 0) {
    const int64_t per_tile = (n_items + p.max_q_tiles - 1) / p.max_q_tiles;  // items as long as one another
    const int64_t tiles = prefix_tiles + (rest + per_tile - 1) / per_tile;   // key tiles of the first of the rest
    const int64_t uneven = rounds % 2 == 1 ? d.sms / per_tile : 0;
    for (int i = 1; i < 4; ++i) {
      const int64_t split = (tiles >> i) + (rounds > 0 ? 8 : 2);
      if (rest <= d.clusters[i] && tiles >> i >= kMinPartTiles && tiles - uneven - split >= 2) shift = i;
    }
  }
  const int64_t whole = shift > 0 ? n_items - rest : n_items;
  cudaLaunchAttribute attr;
  p.first = 0;
  p.by_twos = paired;
  if (!paired && shift == 0 && rounds >= kUnitRounds && p.num_seqs <= kMaxListSeqs && p.max_q_tiles <= kMaxLevels &&
      (p.items ? p.num_items : p.total_q / kBM + p.num_seqs) <= kMaxList && (reinterpret_cast<uintptr_t>(p.out) & 31) == 0) {
    if (p.items)
      prefill_q4_units_kernel<E, true><<<d.sms, kThreads, kUnitsSmemBytes, stream>>>(tq, p);
    else
      prefill_q4_units_kernel<E, false><<<d.sms, kThreads, kUnitsSmemBytes, stream>>>(tq, p);
    return cudaGetLastError();
  }
  if (whole > 0 && paired) {
    const cudaLaunchConfig_t cfg = launch_config(static_cast<unsigned>(whole), 2, &attr, stream);
    e = cudaLaunchKernelEx(&cfg, prefill_q4_kernel<E, Share::kPaired>, tq, const_cast<const Q4PrefillParams&>(p));
    if (e != cudaSuccess) return e;
  } else if (whole > 0) {
    prefill_q4_kernel<E, Share::kWhole><<<static_cast<unsigned>(whole), kThreads, kSmemBytes, stream>>>(tq, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (shift > 0) {
    p.first = static_cast<int32_t>(whole);
    const cudaLaunchConfig_t cfg = launch_config(static_cast<unsigned>(rest) << shift, 1 << shift, &attr, stream);
    return cudaLaunchKernelEx(&cfg, prefill_q4_kernel<E, Share::kSplitKeys>, tq, const_cast<const Q4PrefillParams&>(p));
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_prefill_q4(const void* q, int64_t q_row_stride, int32_t total_q, const void* k_cache,
                              const void* v_cache, int32_t num_blocks, const int32_t* cu_q, const int32_t* cu_k,
                              int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* block_tables,
                              int32_t bt_stride, int32_t num_seqs, int32_t hq, int32_t hkv, float scale,
                              const int32_t* items, int32_t num_items, void* out, unsigned int* err,
                              cudaStream_t stream, Elem elem) {
  CUtensorMap tq;
  if (!encode_q(&tq, q, total_q, hq, q_row_stride, elem)) return cudaErrorInvalidValue;
  Q4PrefillParams p;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.block_tables = block_tables;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.bt_stride = bt_stride;
  p.num_blocks = num_blocks;
  p.num_seqs = num_seqs;
  p.max_q_tiles = (static_cast<int64_t>(max_seqlen_q < total_q ? max_seqlen_q : total_q) + kBM - 1) / kBM;
  p.max_seqlen_q = max_seqlen_q;
  p.max_seqlen_k = max_seqlen_k;
  p.total_q = total_q;
  p.hq = hq;
  p.hkv = hkv;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.items = num_items > 0 ? items : nullptr;
  p.num_items = num_items;
  p.out = static_cast<uint16_t*>(out);
  p.err = err;
  const int64_t pairs = hq / 2;
  const int64_t nblocks = p.items ? num_items * pairs : static_cast<int64_t>(p.max_q_tiles) * num_seqs * pairs;
  if (nblocks > 0x7fffffff) return cudaErrorInvalidValue;
  // tiles of keys before the queries, as far as the bounds of the lengths tell
  const int64_t table_keys = static_cast<int64_t>(bt_stride) * kBlockSize;
  const int64_t keys = max_seqlen_k < table_keys ? max_seqlen_k : table_keys;
  const int64_t queries = max_seqlen_q < total_q ? max_seqlen_q : total_q;
  const int32_t prefix_tiles = keys > queries ? static_cast<int32_t>((keys - queries) / kBN) : 0;
  p.first = 0;
  return elem == Elem::kF16 ? launch_typed<Elem::kF16>(tq, p, nblocks, prefix_tiles, stream)
                            : launch_typed<Elem::kBF16>(tq, p, nblocks, prefix_tiles, stream);
}

}  // namespace pkv
