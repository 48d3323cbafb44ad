// q4_decode.cu -- single-query attention over the 4-bit paged cache (split-KV).
//
// For sequence b, query head h and kv head h / G, with c, s, z the codes,
// scales and minima of q4.cuh (group g of 32 dims):
//   logit_t = scale * sum_g (s_tg * sum_{d in g} q_d c_td + z_tg * sum_{d in g} q_d)
//   out_d   = sum_t p_t (s_tg c_td + z_tg) / sum_t p_t,  p = softmax(logit)
// The codes are used exactly as stored; no 16-bit K or V row is ever formed.
//
// What bounds it: 160 bytes per (token, kv head) from HBM, 47 codes a clock
// and SM at the copy rate. Widening and multiplying them on the CUDA cores
// (an unpack and two multiply-adds per code and query head) would need more
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
//    G = 4 query heads take a second B; A is widened once.
//  * p goes from C's layout to B's by movmatrix (8 x 8 transpose in registers).
//  * q is scaled by a power of two per head so that fp16 holds it exactly
//    (elements below 2^-38 of the head's largest are rounded); p s is scaled by
//    a running power of two and rounded to fp16 (relative 2^-11, as p is in any
//    tensor-core product). Sums, maxima and the z terms stay in fp32.
//
// Work: an item is a chunk of up to 256 tokens of one (sequence, kv head), and
// a warp works through items alone: it fetches 32 tokens a stage by two bulk
// copies (K and V tiles of one (block, head) are contiguous) into its own ring
// in shared memory and waits on its own barriers, so no warp ever waits for
// another. One CTA of kWarps warps per SM. Every CTA derives the item table
// from context_lens; warp w starts on item w and takes the next ones from a
// counter in the workspace. Partial results (m, l, o) of sequences with several
// chunks go to the workspace, and the warp that finishes last merges them
// (ticket, no waiting): up to 16 chunks at once, groups of 16 and then the
// groups beyond that.
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

constexpr int kUnit = 32;                                    // tokens per stage
constexpr int kUnitTiles = kUnit / kQ4Tile;
constexpr int kUnitBytes = kUnitTiles * kQ4TileBytes;        // 2560, of K and of V each
constexpr int kMaxChunk = kBlockSize / kUnit;                // units per item at most
constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kMaxSeqs = 1024;                               // sequences per launch (item table in shared memory)
constexpr int kPlanWarps = 152 * kWarps;                     // warps the chunk rule splits a call over
constexpr int kFan = 16;                                     // chunks merged at once

struct Q4DecodeParams {
  const uint16_t* q;
  int64_t q_row_stride;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  int32_t num_blocks;
  int32_t hkv;
  const int32_t* block_tables;
  int32_t bt_stride;
  const int32_t* context_lens;
  int32_t max_ctx;
  int32_t num_seqs;
  float scale_log2;
  uint16_t* out;
  int32_t* work;     // {next item, warps done}, zero between calls
  int32_t* tickets;  // one per item, zero between calls
  float2* ml;        // [item][G] (max in log2 units, sum)
  float* opart;      // [item][G][128], not normalised
  int64_t max_items;
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

// Units per chunk. x is the number of units each planned warp would get: up to
// kMaxChunk, one chunk each; beyond, as many rounds of equal chunks as keep a
// chunk within kMaxChunk.
__host__ __device__ inline int chunk_units(int64_t units_all_heads) {
  const int64_t x = (units_all_heads + kPlanWarps - 1) / kPlanWarps;
  if (x <= 1) return 1;
  const int64_t rounds = (x + kMaxChunk - 1) / kMaxChunk;
  return static_cast<int>((x + rounds - 1) / rounds);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr));
  return r;
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

// Merges n partials (slots first, first + stride, ...) of one query head, 4 dims
// per lane: o = sum 2^(m - M) o_i, l = sum 2^(m - M) l_i, M the largest m.
__device__ __forceinline__ void merge_slots(const Q4DecodeParams& p, int64_t first, int64_t stride, int n, int G, int h,
                                            int lane, float& M, float& den, float4& acc) {
  constexpr int kAhead = 4;  // the partials sit in L2: loads of four slots in flight
  M = -INFINITY;
  den = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = 0; c0 < n; c0 += kAhead) {
    float2 ml[kAhead];
    float4 o[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c0 + i < n) {
        const int64_t slot = (first + (c0 + i) * stride) * G + h;
        ml[i] = __ldcg(p.ml + slot);
        o[i] = __ldcg(reinterpret_cast<const float4*>(p.opart + slot * kHeadDim) + lane);
      }
    }
    float Mg = M;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) Mg = fmaxf(Mg, ml[i].x);
    const float Mu = (Mg == -INFINITY) ? 0.f : Mg;
    const float sc = ex2_approx(M - Mu);
    M = Mg;
    den *= sc;
    acc.x *= sc;
    acc.y *= sc;
    acc.z *= sc;
    acc.w *= sc;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float w = ex2_approx(ml[i].x - Mu);
      den = fmaf(w, ml[i].y, den);
      acc.x = fmaf(w, o[i].x, acc.x);
      acc.y = fmaf(w, o[i].y, acc.y);
      acc.z = fmaf(w, o[i].z, acc.z);
      acc.w = fmaf(w, o[i].w, acc.w);
    }
  }
}

template <Elem E, int G>
__global__ void __launch_bounds__(kThreads, 1) q4_decode_kernel(const Q4DecodeParams p) {
  using Ops = ElemOps<E>;
  constexpr int kNB = (G + 1) / 2;            // B operands: pairs of query heads
  constexpr int kQBytes = G * kHeadDim * 2;   // one item's query rows
  constexpr int kStageBytes = 2 * kUnitBytes + kQBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  int4* hdr_all = reinterpret_cast<int4*>(smem + kWarps * kStages * kStageBytes);  // [warp][stage]
  uint64_t* bars = reinterpret_cast<uint64_t*>(hdr_all + kWarps * kStages);        // [warp][stage]
  int* sF = reinterpret_cast<int*>(bars + kWarps * kStages);                       // [num_seqs + 1] chunks before b
  int* sCtx = sF + kMaxSeqs + 1;                                                   // [num_seqs]
  int* red = sCtx + kMaxSeqs;                                                      // [kWarps]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.num_seqs;
  const int n_ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);

  // ---- item table: chunks before each sequence ----
  int chunk;  // units per chunk
  {
    constexpr int kPer = (kMaxSeqs + kThreads - 1) / kThreads;
    const int per = (B + kThreads - 1) / kThreads;  // consecutive sequences per thread
    int ctx[kPer];
    int units = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * per + i;
      ctx[i] = 0;
      if (i < per && b < B) {
        const int c = p.context_lens[b];
        if (c < 0 || c > p.max_ctx || c > static_cast<int64_t>(p.bt_stride) * kBlockSize) {
          if (cta == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
        } else {
          ctx[i] = c;
        }
        sCtx[b] = ctx[i];
      }
      units += (ctx[i] + kUnit - 1) / kUnit;
    }
    int sum = units;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) red[warp] = sum;
    if (lane < kStages) mbar_init(smem_u32(bars + warp * kStages + lane), 1);
    mbar_fence_init();
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += red[w];
    chunk = chunk_units(all * p.hkv);
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += ((ctx[i] + kUnit - 1) / kUnit + chunk - 1) / chunk;
    int scan = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, off);
      if (lane >= off) scan += y;
    }
    __syncthreads();  // every thread has read red
    if (lane == 31) red[warp] = scan;
    __syncthreads();
    int before = scan - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (w < warp) before += red[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * per + i;
      if (i < per && b < B) {
        sF[b] = before;
        before += ((ctx[i] + kUnit - 1) / kUnit + chunk - 1) / chunk;
        if (b == B - 1) sF[B] = before;
      }
    }
    __syncthreads();
  }
  const int64_t n_items = static_cast<int64_t>(sF[B]) * p.hkv;
  if (n_items > p.max_items) {  // cannot happen: the workspace bound covers every table
    if (tid == 0) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
    return;
  }

  // rows without context: zeros
  for (int b = cta * kWarps + warp; b < B; b += n_ctas * kWarps) {
    if (sCtx[b] == 0) {
      uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(b) * p.hkv * G * kHeadDim);
      for (int i = lane; i < p.hkv * G * (kHeadDim / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
    }
  }

  const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes;
  const uint32_t full = smem_u32(bars + warp * kStages);
  int4* hdr = hdr_all + warp * kStages;
  const int r = lane >> 2, t = lane & 3;
  const int W = n_ctas * kWarps;
  const bool dynamic = n_items > W;

  // ---- the issuing side: which unit is fetched next ----
  int64_t item = static_cast<int64_t>(warp) * n_ctas + cta;
  int next_raw = 0;  // lane 0: the counter's answer for the item after this one
  if (dynamic && lane == 0) next_raw = atomicAdd(p.work, 1);
  int ib = 0, ihead = 0, ic = 0, inch = 0, iu = 0, iend = 0, ipb = -1, ipblk = -1;
  auto resolve = [&]() {  // item -> sequence, chunk, head (whole warp)
    const int ci = static_cast<int>(item / p.hkv);
    ihead = static_cast<int>(item - static_cast<int64_t>(ci) * p.hkv);
    // largest b with sF[b] <= ci, 32 probes at a time
    const int step = (B + 31) / 32;
    const int probe = lane * step;
    const int hi = __popc(__ballot_sync(0xffffffffu, probe < B && sF[probe] <= ci)) - 1;
    const int q0 = hi * step;
    const int probe2 = q0 + lane;
    const int cnt = __popc(__ballot_sync(0xffffffffu, lane < step && probe2 < B && sF[probe2] <= ci));
    ib = q0 + cnt - 1;
    ic = ci - sF[ib];
    inch = sF[ib + 1] - sF[ib];
    iu = ic * chunk;
    iend = min(iu + chunk, (sCtx[ib] + kUnit - 1) / kUnit);
    ipblk = -1;
  };
  bool more = item < n_items;
  if (more) resolve();
  int issued = 0;
  auto issue = [&]() {  // fetches one unit into slot issued % kStages (whole warp)
    if (!more) return;
    const int s = issued % kStages;
    const int ctx = sCtx[ib];
    const int tok0 = iu * kUnit;
    const int ntok = min(kUnit, ctx - tok0);
    if (ipblk != tok0 / kBlockSize) {
      ipblk = tok0 / kBlockSize;
      ipb = p.block_tables[static_cast<int64_t>(ib) * p.bt_stride + ipblk];
      if (ipb < 0 || ipb >= p.num_blocks) {
        if (lane == 0) flag_error(p.err, PKV_DEVERR_BAD_BLOCK);
        ipb = -1;
      }
    }
    const int64_t rec = (static_cast<int64_t>(ipb) * p.hkv + ihead) * kQ4RecordBytes;
    const bool last = iu + 1 == iend;
    if (p.k_new != nullptr && last && ic == inch - 1) {
      // this unit holds the newest position: its row is written before the unit is fetched
      const int64_t slot = p.slot_mapping[ib];
      if (slot != -1) {
        if (ipb < 0 || slot != static_cast<int64_t>(ipb) * kBlockSize + (ctx - 1) % kBlockSize) {
          if (lane == 0 && ihead == 0) flag_error(p.err, PKV_DEVERR_BAD_SLOT);
        } else {
          const int lane16 = lane & 15, j = lane16 >> 2, tt = lane16 & 3;
          const bool is_v = lane >= 16;
          const uint16_t* src = (is_v ? p.v_new + ib * p.v_new_stride : p.k_new + ib * p.k_new_stride) +
                                ihead * kHeadDim + lane16 * 8;
          uint32_t par;
          uint32_t codes = quantise8<E>(*reinterpret_cast<const uint4*>(src), par);
          const uint32_t vcodes = v_exchange(codes, j);
          const int in_block = (ctx - 1) % kBlockSize, tok = in_block % kQ4Tile;
          uint8_t* dst = (is_v ? p.v_cache_w : p.k_cache_w) + rec + in_block / kQ4Tile * kQ4TileBytes;
          *reinterpret_cast<uint32_t*>(dst + (is_v ? q4_v_word(tok, j, tt) : q4_k_word(tok, j, tt))) =
              is_v ? vcodes : codes;
          if (tt == 0) *reinterpret_cast<uint32_t*>(dst + q4_param(tok, j)) = par;
          // visible to the bulk copy (async proxy) that lane 0 issues below
          asm volatile("fence.proxy.async.global;" ::: "memory");
          __syncwarp();
        }
      }
    }
    if (lane == 0) {
      const uint32_t dst = ring + s * kStageBytes;
      const bool first = iu == ic * chunk;
      const uint32_t bytes = ipb < 0 ? 0u : static_cast<uint32_t>((ntok + kQ4Tile - 1) / kQ4Tile) * kQ4TileBytes;
      hdr[s] = make_int4(ib, ihead | (static_cast<int>(first) << 30) | (static_cast<int>(last) << 29),
                         ipb < 0 ? 0 : ntok, ic);
      mbar_arrive_expect_tx(full + 8 * s, 2 * bytes + (first ? kQBytes : 0));
      if (bytes > 0) {
        const int64_t off = rec + (tok0 % kBlockSize) / kQ4Tile * kQ4TileBytes;
        bulk_g2s(dst, p.k_cache + off, bytes, full + 8 * s);
        bulk_g2s(dst + kUnitBytes, p.v_cache + off, bytes, full + 8 * s);
      }
      if (first)
        bulk_g2s(dst + 2 * kUnitBytes, p.q + static_cast<int64_t>(ib) * p.q_row_stride + ihead * G * kHeadDim, kQBytes,
                 full + 8 * s);
    }
    ++issued;
    ++iu;
    if (last) {
      more = false;
      if (dynamic) {
        item = static_cast<int64_t>(W) + __shfl_sync(0xffffffffu, next_raw, 0);
        more = item < n_items;
        if (more) {
          if (lane == 0) next_raw = atomicAdd(p.work, 1);
          resolve();
        }
      }
    }
  };
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) issue();

  // ---- the computing side ----
  // lane (r, t): K rows (C fragment) of tokens tk, tk + 8 and group t; V columns
  // of tokens tv, tv ^ 1, tv + 8, (tv ^ 1) + 8 and 16-dim chunk r. Row r of a C
  // fragment stands for token r ^ (r >> 1 & 1), which makes both loads free of
  // bank conflicts.
  const int tk = r ^ ((r >> 1) & 1);
  const int tv = (2 * t) ^ (t & 1);
  const uint32_t k_off = tk * kQ4CodeBytes + t * 16;
  const uint32_t par_off = kQ4TileParams + tk * kQ4ParamBytes + t * 4;
  const uint32_t va_off = tv * kQ4CodeBytes + ((r ^ (tv & 4)) << 3);
  const uint32_t vb_off = (tv ^ 1) * kQ4CodeBytes + ((r ^ (tv & 4)) << 3);
  uint32_t qb[kNB][8][2];           // B fragments of q, one per 16 dims
  float kc[G + (G & 1)], qs[G + (G & 1)];
  float acc[kNB][8][4];
  float m[G], l[G], zs[G];
  float nu = 1.f;
  int done = 0;
  for (; done < issued; ++done) {
    const int s = done % kStages;
    if (!__all_sync(0xffffffffu, mbar_wait(full + 8 * s, (done / kStages) & 1, p.err))) break;
    const int4 hd = hdr[s];
    const uint32_t st = ring + s * kStageBytes;
    if (hd.y & (1 << 30)) {
      // ---- a new item: query fragments ----
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) {
        const int h = 2 * nb + (r & 1);  // the column's head; its group is r >> 1
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (h < G) raw = lds128(st + 2 * kUnitBytes + h * kHeadDim * 2 + ((r >> 1) * 32 + t * 8) * 2);
        float x[8] = {Ops::lo(raw.x), Ops::hi(raw.x), Ops::lo(raw.y), Ops::hi(raw.y),
                      Ops::lo(raw.z), Ops::hi(raw.z), Ops::lo(raw.w), Ops::hi(raw.w)};
        float big = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          big = fmaxf(big, fabsf(x[i]));
          sum += x[i];
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 8));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 16));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int e = big > 0.f ? max(-100, 13 - exponent_of(big)) : 0;  // the largest |q| goes to [2^13, 2^14)
        const float f = pow2(min(e, 120));
        const float f16 = f * 0.0625f;  // for the codes that A holds 16 times too large
        const uint32_t own[4] = {pack_f16(x[0] * f, x[4] * f), pack_f16(x[1] * f16, x[5] * f16),
                                 pack_f16(x[2] * f, x[6] * f), pack_f16(x[3] * f16, x[7] * f16)};
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const bool on = (ks >> 1) == (r >> 1);
          qb[nb][ks][0] = on ? own[(ks & 1) * 2] : 0u;
          qb[nb][ks][1] = on ? own[(ks & 1) * 2 + 1] : 0u;
        }
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const float fh = __shfl_sync(0xffffffffu, f, 4 * h2);
          kc[2 * nb + h2] = __fdividef(16777216.f, fh) * p.scale_log2;  // a power of two times scale * log2(e)
          qs[2 * nb + h2] = __shfl_sync(0xffffffffu, sum, (2 * t + h2) * 4) * p.scale_log2;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[nb][i][c] = 0.f;
      }
#pragma unroll
      for (int h = 0; h < G; ++h) {
        m[h] = -INFINITY;
        l[h] = zs[h] = 0.f;
      }
      nu = 1.f;
    }
    const int ntok = hd.z;
    if (ntok > 0) {
      // ---- logits ----
      float lg[kNB][kUnitTiles][4];  // [2 half + head]: token tk + 8 half
#pragma unroll
      for (int tile = 0; tile < kUnitTiles; ++tile) {
        const uint32_t base = st + tile * kQ4TileBytes;
        const uint4 w0 = lds128(base + k_off), w1 = lds128(base + k_off + 8 * kQ4CodeBytes);
        const float2 sz0 = h2_to_f2(lds32(base + par_off)), sz1 = h2_to_f2(lds32(base + par_off + 8 * kQ4ParamBytes));
        float c[kNB][4];
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) c[nb][0] = c[nb][1] = c[nb][2] = c[nb][3] = 0.f;
        const uint32_t a[4] = {w0.x, w0.y, w0.z, w0.w}, b[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t ah = a[j] >> 8, bh = b[j] >> 8;
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) {
            mma16816(c[nb], a[j] & 0x000f000fu, b[j] & 0x000f000fu, a[j] & 0x00f000f0u, b[j] & 0x00f000f0u,
                     qb[nb][2 * j][0], qb[nb][2 * j][1]);
            mma16816(c[nb], ah & 0x000f000fu, bh & 0x000f000fu, ah & 0x00f000f0u, bh & 0x00f000f0u,
                     qb[nb][2 * j + 1][0], qb[nb][2 * j + 1][1]);
          }
        }
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            float x0 = fmaf(c[nb][h2], sz0.x * kc[2 * nb + h2], sz0.y * qs[2 * nb + h2]);
            float x1 = fmaf(c[nb][2 + h2], sz1.x * kc[2 * nb + h2], sz1.y * qs[2 * nb + h2]);
            x0 += __shfl_xor_sync(0xffffffffu, x0, 1);
            x1 += __shfl_xor_sync(0xffffffffu, x1, 1);
            x0 += __shfl_xor_sync(0xffffffffu, x0, 2);
            x1 += __shfl_xor_sync(0xffffffffu, x1, 2);
            lg[nb][tile][h2] = x0;
            lg[nb][tile][2 + h2] = x1;
          }
      }
      // V's scale and minimum of this lane's tokens and group; past the end both are 0
      float2 vsz[kUnitTiles][2];
#pragma unroll
      for (int tile = 0; tile < kUnitTiles; ++tile)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const bool in = tile * kQ4Tile + 8 * half + tk < ntok;
          const uint32_t w = lds32(st + kUnitBytes + tile * kQ4TileBytes + par_off + half * 8 * kQ4ParamBytes);
          vsz[tile][half] = h2_to_f2(in ? w : 0u);
          if (!in) {
#pragma unroll
            for (int nb = 0; nb < kNB; ++nb) lg[nb][tile][2 * half] = lg[nb][tile][2 * half + 1] = -INFINITY;
          }
        }
      // ---- running maximum: moves only when a logit passes it by more than 8 (2^8 of headroom) ----
      float top[G];
      bool moved = false;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float x = -INFINITY;
#pragma unroll
        for (int tile = 0; tile < kUnitTiles; ++tile)
          x = fmax3(x, lg[h / 2][tile][h & 1], lg[h / 2][tile][2 + (h & 1)]);
        top[h] = x;
        moved |= x > m[h] + 8.f;
      }
      moved = __any_sync(0xffffffffu, moved);
      if (moved) {
#pragma unroll
        for (int h = 0; h < G; ++h) {
          float x = top[h];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(x, m[h]);
          const float sc = ex2_approx(m[h] - (x == -INFINITY ? 0.f : x));
          m[h] = x;
          l[h] *= sc;
          zs[h] *= sc;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[h / 2][i][h & 1] *= sc;
            acc[h / 2][i][2 + (h & 1)] *= sc;
          }
        }
      }
      // ---- p, its sums, and p * s for the product with V's codes ----
      float w[kNB][kUnitTiles][4];
      float wmax = 0.f;
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
        for (int tile = 0; tile < kUnitTiles; ++tile)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int h = 2 * nb + (i & 1);
            w[nb][tile][i] = 0.f;
            if (h < G) {
              const float mu = m[h] == -INFINITY ? 0.f : m[h];
              const float pr = ex2_approx(lg[nb][tile][i] - mu);
              l[h] += pr;
              zs[h] = fmaf(pr, vsz[tile][i >> 1].y, zs[h]);
              w[nb][tile][i] = pr * vsz[tile][i >> 1].x;
              wmax = fmaxf(wmax, w[nb][tile][i]);
            }
          }
      if (moved || __any_sync(0xffffffffu, wmax * nu > 16384.f)) {
        // nu: the power of two that takes the largest p s of this unit to [1, 2)
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, off));
        const float nu2 = pow2(max(-24, min(24, -exponent_of(wmax))));
        const float sc = __fdividef(nu2, nu);
        nu = nu2;
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[nb][i][c] *= sc;
      }
      // ---- o += (p s) . V codes ----
#pragma unroll
      for (int tile = 0; tile < kUnitTiles; ++tile) {
        uint32_t pb[kNB][2];
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) {
          pb[nb][0] = movmatrix(pack_f16(w[nb][tile][0] * nu, w[nb][tile][1] * nu));
          pb[nb][1] = movmatrix(pack_f16(w[nb][tile][2] * nu, w[nb][tile][3] * nu));
        }
        const uint32_t base = st + kUnitBytes + tile * kQ4TileBytes;
        const uint2 a0 = lds64(base + va_off), a1 = lds64(base + vb_off);
        const uint2 b0 = lds64(base + va_off + 8 * kQ4CodeBytes), b1 = lds64(base + vb_off + 8 * kQ4CodeBytes);
        const uint32_t lo[4] = {__byte_perm(a0.x, a1.x, 0x5410), __byte_perm(a0.x, a1.x, 0x7632),
                                __byte_perm(a0.y, a1.y, 0x5410), __byte_perm(a0.y, a1.y, 0x7632)};
        const uint32_t hi[4] = {__byte_perm(b0.x, b1.x, 0x5410), __byte_perm(b0.x, b1.x, 0x7632),
                                __byte_perm(b0.y, b1.y, 0x5410), __byte_perm(b0.y, b1.y, 0x7632)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo8 = lo[j] >> 8, hi8 = hi[j] >> 8;
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) {
            mma16816(acc[nb][2 * j], lo[j] & 0x000f000fu, lo[j] & 0x00f000f0u, hi[j] & 0x000f000fu,
                     hi[j] & 0x00f000f0u, pb[nb][0], pb[nb][1]);
            mma16816(acc[nb][2 * j + 1], lo8 & 0x000f000fu, lo8 & 0x00f000f0u, hi8 & 0x000f000fu,
                     hi8 & 0x00f000f0u, pb[nb][0], pb[nb][1]);
          }
        }
      }
    }
    __syncwarp();  // every lane has read the slot
    issue();
    if (!(hd.y & (1 << 29))) continue;

    // ---- the item's end: dims 32 t + 4 r .. + 3 of every head in this lane ----
    const int b = hd.x, head = hd.y & 0xffff, c = hd.w;
    const int first_chunk = sF[b], nch = sF[b + 1] - first_chunk;
    const int64_t slot = static_cast<int64_t>(first_chunk + c) * p.hkv + head;
    uint16_t* orow = p.out + (static_cast<int64_t>(b) * p.hkv + head) * G * kHeadDim;
    const float back = __fdividef(16777216.f, nu);
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float sum = l[h], z = zs[h];
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
        z += __shfl_xor_sync(0xffffffffu, z, off);
      }
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int f = (i >> 1), cc = (i & 1) * 2 + (h & 1);
        float x = acc[h / 2][f][cc];
        x = t == 1 ? acc[h / 2][2 + f][cc] : x;
        x = t == 2 ? acc[h / 2][4 + f][cc] : x;
        x = t == 3 ? acc[h / 2][6 + f][cc] : x;
        o[i] = fmaf(x, (i & 1) ? back * 0.0625f : back, z);
      }
      const int d = 32 * t + 4 * r;
      if (nch == 1) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint2 v;
        v.x = Ops::pack(o[0] * inv, o[1] * inv);
        v.y = Ops::pack(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2*>(orow + h * kHeadDim + d) = v;
      } else {
        *reinterpret_cast<float4*>(p.opart + (slot * G + h) * kHeadDim + d) = make_float4(o[0], o[1], o[2], o[3]);
        if (lane == 0) p.ml[slot * G + h] = make_float2(m[h], sum);
      }
    }
    if (nch == 1) continue;

    // ---- merge by the warp that finishes last ----
    auto arrive = [&](int64_t at, int expected) -> bool {
      __threadfence();
      __syncwarp();
      int last = 0;
      if (lane == 0) {
        last = atomicAdd(p.tickets + at, 1) == expected - 1;
        if (last) p.tickets[at] = 0;  // ready for the next call
      }
      last = __shfl_sync(0xffffffffu, last, 0);
      if (last) __threadfence();
      return last != 0;
    };
    const int g0 = c - c % kFan;  // this chunk's group of kFan
    const int64_t slot_g = static_cast<int64_t>(first_chunk + g0) * p.hkv + head;
    const int in_group = min(kFan, nch - g0);
    if (!arrive(slot_g, in_group)) continue;
    int64_t from = slot_g, stride = p.hkv;
    int n = in_group;
    if (nch > kFan) {
      // merge the group into its first slot, then the groups
#pragma unroll 1
      for (int h = 0; h < G; ++h) {
        float M, den;
        float4 a;
        merge_slots(p, slot_g, p.hkv, in_group, G, h, lane, M, den, a);
        reinterpret_cast<float4*>(p.opart + (slot_g * G + h) * kHeadDim)[lane] = a;
        __syncwarp();
        if (lane == 0) p.ml[slot_g * G + h] = make_float2(M, den);
      }
      const int groups = (nch + kFan - 1) / kFan;
      const int64_t slot_0 = static_cast<int64_t>(first_chunk) * p.hkv + head;
      if (!arrive(slot_0 + p.hkv, groups)) continue;  // the ticket of chunk 1, which no group uses
      from = slot_0;
      stride = static_cast<int64_t>(kFan) * p.hkv;
      n = groups;
    }
#pragma unroll 1
    for (int h = 0; h < G; ++h) {
      float M, den;
      float4 a;
      merge_slots(p, from, stride, n, G, h, lane, M, den, a);
      const float inv = den == 0.f ? 0.f : 1.f / den;
      uint2 v;
      v.x = Ops::pack(a.x * inv, a.y * inv);
      v.y = Ops::pack(a.z * inv, a.w * inv);
      reinterpret_cast<uint2*>(orow + h * kHeadDim)[lane] = v;
    }
  }
  // only after a wait that ran out: never leave a copy in flight into this CTA's shared memory
  for (; done < issued; ++done) mbar_wait(full + 8 * (done % kStages), (done / kStages) & 1, p.err);

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
  return static_cast<size_t>(kWarps) * kStages * (2 * kUnitBytes + G * kHeadDim * 2 + sizeof(int4) + sizeof(uint64_t)) +
         (2 * kMaxSeqs + 1 + kWarps) * sizeof(int);
}
static_assert(smem_bytes<4>() <= 227 * 1024, "shared memory above the 227 KB a CTA can opt into");

template <Elem E, int G>
cudaError_t launch_typed(const Q4DecodeParams& p, cudaStream_t stream) {
  static bool attr_done[64] = {false};
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(q4_decode_kernel<E, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem_bytes<G>()));
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) sms = 152;
  q4_decode_kernel<E, G><<<sms, kThreads, smem_bytes<G>(), stream>>>(p);
  return cudaGetLastError();
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Most items that a launch over these sizes can have. chunk_units gives one
// item per planned warp up to x = kMaxChunk units each, chunks of at least 5
// units for x <= 64 and of kMaxChunk beyond, plus one short chunk per sequence
// and head; and never more items than units.
int64_t max_items(int64_t num_seqs, int64_t hkv, int64_t max_ctx) {
  const int64_t units = num_seqs * ((max_ctx + kUnit - 1) / kUnit) * hkv;
  int64_t chunks = int64_t{64} * kPlanWarps / 5 + 1;
  if (units / kMaxChunk + 1 > chunks) chunks = units / kMaxChunk + 1;
  chunks += num_seqs * hkv;
  return units < chunks ? units : chunks;
}

}  // namespace

// Workspace: two work counters and a ticket per item (zero between calls), then
// the items' partial outputs and (m, l). Launches of kMaxSeqs sequences follow
// one another on the stream and share it. The counters' region depends on the
// size of the workspace alone, so that calls of other sizes on the same
// workspace find zeros there: 1/128 of it, which holds the tickets (4 bytes) of
// any number of items (520 bytes or more) that fit in the rest.
size_t decode_q4_counter_bytes(size_t workspace_bytes) { return 256 + (workspace_bytes / 128 & ~size_t{255}); }

size_t decode_q4_workspace_bytes(int32_t num_seqs, int32_t hkv, int32_t group, int32_t max_ctx) {
  const int64_t n = max_items(num_seqs < kMaxSeqs ? num_seqs : kMaxSeqs, hkv, max_ctx);
  const size_t partials = static_cast<size_t>(n) * group * (kHeadDim * sizeof(float) + sizeof(float2));
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
    const int64_t n = max_items(num_seqs < kMaxSeqs ? num_seqs : kMaxSeqs, hkv, max_ctx);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.work = reinterpret_cast<int32_t*>(ws);
    p.tickets = p.work + 2;
    ws += decode_q4_counter_bytes(workspace_bytes);
    p.opart = reinterpret_cast<float*>(ws);
    p.ml = reinterpret_cast<float2*>(ws + static_cast<size_t>(n) * group * kHeadDim * sizeof(float));
    p.max_items = n;
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
    cudaError_t e = cudaErrorInvalidValue;
    const bool f16 = elem == Elem::kF16;
    if (group == 1)
      e = f16 ? launch_typed<Elem::kF16, 1>(p, stream) : launch_typed<Elem::kBF16, 1>(p, stream);
    else if (group == 2)
      e = f16 ? launch_typed<Elem::kF16, 2>(p, stream) : launch_typed<Elem::kBF16, 2>(p, stream);
    else if (group == 4)
      e = f16 ? launch_typed<Elem::kF16, 4>(p, stream) : launch_typed<Elem::kBF16, 4>(p, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pkv
