// decode_mod.cu -- single-query attention over the paged cache whose scores are capped, biased by distance or see a part
// of the keys, for any head counts; and each key's attention added up beside it.
//
// For sequence b with p = context_lens[b] - 1, query head h, kv head h / G and every visible t (start_b <= t <= p and
// p - t < window):
//   x_t = scale * q . k_t;   s_t = cap * tanh(x_t / cap) (or x_t);   z_t = s_t - slope_h * (p - t)
//   out = sum_t e^(z_t - m) v_t / sum_t e^(z_t - m),    weights[t] += sum over the G heads of a kv head of their share.
//
// What bounds it: 512 bytes of K and V per (token, kv head) from HBM: 256 sequences of 512..4096 tokens, 16 heads on 8,
// with weights 404 us, the main kernel 383 of them at 0.95 of a plain copy's rate; one of 40007, 32 on 8, 36.8 us, 20 of
// them streaming, the others the start (scan of the lengths, first table entries, first copies) and the joins. The
// products run on mma.sync m16n8k16 with the
// tokens as rows: S^T = K Q^T for up to 8 query heads of a kv head at a time (their number changes nothing but the
// columns in use), O^T += V^T P. tcgen05 would work on 128 rows of which a kv head has 1 to 16; as it is, the two
// products of 16 tokens and one kv head are 24 instructions where HBM takes 380 clocks for their 8 KB. That leaves time
// for exact arithmetic: p goes to the second product as two 16-bit parts (p and what its rounding lost), tanhf is CUDA's.
//
// Work: a warp is a worker of its own. Each (kv head, part of its query heads) is a stream; a stream's units, 16 tokens
// of a sequence each, are laid end to end and cut into R equal ranges, so that every worker gets the same number of
// bytes, whatever the lengths. Workers of one CTA take the same range of neighbouring heads: their rows lie side by
// side. Every CTA derives the ranges from context_lens; nothing is kept from one call for the next. A worker's 16-token
// units of K and of V come by TMA (two 128-byte halves of each row, 128-byte swizzle) into a ring of kStages of its
// own, and it waits on its own barriers. The reference (the running maximum; of fp16 rows 2^7 below it, see kLift) only
// moves when a score passes it by 2^8, so a step needs one vote and no shuffles.
// A sequence that ends inside the range in which it began is written out at once. For the others the workers leave
// (max, sum, o) in the workspace and a second kernel joins them in order; with weights a third one turns the scores,
// which the first left in the workspace, into shares. Equal calls give equal bits.
#include <atomic>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include <cuda.h>

#include "pkv_common.cuh"

namespace pkv {

struct DecodeModArgs {
  const void* q;
  int64_t q_row_stride;
  const void* k_cache;
  const void* v_cache;
  int32_t num_blocks;
  const int32_t* block_tables;
  int32_t bt_stride;
  const int32_t* context_lens;
  int32_t num_seqs, hq, hkv, max_ctx;
  float scale, softcap;
  const float* slopes;
  int32_t window;
  const int32_t* key_starts;
  float* weights;
  void* out;
  void* workspace;
};

namespace {

constexpr int kUnit = 16;                           // tokens
constexpr int kUnitBytes = kUnit * kHeadDim * 2;    // 4 KB, of K and of V each
constexpr int kStages = 3;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtas = 152;                          // one to an SM
constexpr int kWorkers = kCtas * kWarps;
constexpr int kMinUnits = 2;                        // units to a range at least
constexpr int kOffBars = kWarps * kStages * 2 * kUnitBytes;
constexpr int kOffScan = kOffBars + kWarps * kStages * 8;
constexpr int kOffPieces = kOffScan + (kThreads + kWarps) * 8;
// What a worker has of a sequence that is not all in its range, for the other workers of the CTA.
struct Piece {
  int32_t seq;         // -1: none
  int32_t ends;        // its last unit is here
  int64_t first_unit;  // the sequence's first unit, and the one behind its last
  int64_t end_unit;
  const float2* ml;    // (max, sum) and o per head: in the worker's ring, or in the workspace if that was still in use
  const float* o;
};
constexpr int kPieces = 2 * kWarps;
constexpr size_t kSmemBytes = kOffPieces + kPieces * sizeof(Piece) + 1024;  // + alignment slack
constexpr int kMergeWarps = 16;
constexpr float kLog2e = 1.4426950408889634f;
// A row's largest share before it is divided by their sum, log2: fp16 shares go down to 2^-24 in steps of as much, two
// parts together too, so this much more of the small ones is kept (and 2^7 with 2^8 of headroom stays below fp16's largest
// number).
template <Elem E>
constexpr float kLift = E == Elem::kF16 ? 7.f : 0.f;
constexpr float kNoCap = 1e30f;  // from here on a cap changes no score that fp32 tells from its neighbours below 1e26

// How a call's heads are cut into streams: parts of up to 8 or 16 query heads of one kv head.
struct Streams {
  int32_t group, per, heads, parts, count, ranges;  // heads: of the largest part
  int32_t by_cta;  // a CTA's workers share a stream, and their partial results are joined before they leave the CTA
};
Streams streams_of(int32_t hq, int32_t hkv, int32_t num_seqs, int32_t max_ctx) {
  Streams s;
  s.group = hq / hkv;
  s.per = s.group <= 8 ? 8 : 16;
  s.heads = s.group < s.per ? s.group : s.per;
  s.parts = (s.group + s.per - 1) / s.per;
  s.count = hkv * s.parts;
  s.ranges = s.count < kWorkers ? kWorkers / s.count : 1;
  // Two ways to share the streams out. Workers take them in turn: neighbouring heads' rows, which lie side by side, are
  // read at the same time, but each of a long sequence's pieces goes through memory (256 sequences: 409 us, the other way
  // 418). Or a CTA takes eight neighbouring ranges of one stream and joins its workers' pieces (one sequence of 40007,
  // 32 on 8 heads: 37.0 us instead of 38.2; 14 of up to 1000, 12 heads: 23.6, 24.4): for short ranges, and where the
  // streams leave at most one CTA in 16 over.
  const int32_t ctas = kCtas / s.count;
  const int64_t units = (static_cast<int64_t>(max_ctx) + kUnit - 1) / kUnit * num_seqs;
  s.by_cta = ctas * s.count * 16 >= kCtas * 15 && units <= 128 * s.ranges;
  if (s.by_cta) s.ranges = ctas * kWarps;
  return s;
}

// Workspace: RangeInfo per range, (max, 1 / sum) per (sequence, query head), partial (max, sum) and o per (range, stream,
// first or last sequence of the range, head of the part), and with weights the scores per (sequence, unit, stream, head
// of the part, token).
struct alignas(16) RangeInfo {  // the sequence that begins in this range and goes on behind it
  int32_t seq;         // -1: none
  int32_t last;        // the range that holds its last unit
  int32_t place;       // its partial results are this range's first (0) or last (1); in later ranges they are the first
  int32_t pad;
};
struct Layout {
  size_t info, final_ml, ml, o, scores, total;
};
Layout layout_of(const Streams& s, int32_t num_seqs, int32_t hq, int32_t max_ctx, bool weights) {
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 127) / 128 * 128;
    return here;
  };
  const size_t slots = static_cast<size_t>(s.ranges) * s.count * 2 * s.heads;
  l.info = take(sizeof(RangeInfo) * s.ranges);
  l.final_ml = take(weights ? sizeof(float2) * num_seqs * hq : 0);
  l.ml = take(sizeof(float2) * slots);
  l.o = take(sizeof(float) * kHeadDim * slots);
  const size_t units = (static_cast<size_t>(max_ctx) + kUnit - 1) / kUnit;
  l.scores = take(weights ? sizeof(float) * num_seqs * units * s.count * s.heads * kUnit : 0);
  l.total = at;
  return l;
}

struct DecodeModParams {
  const uint16_t* q;
  int64_t q_row_stride;
  const uint16_t* v;  // the cache once more, for values that are not finite
  const int32_t* block_tables;
  int32_t bt_stride, num_blocks;
  const int32_t* context_lens;
  int32_t num_seqs, hq, hkv, max_ctx;
  Streams st;
  float scale_log2, cap_log2, scale_by_cap;  // cap_log2 == 0: no cap
  const float* slopes;
  int32_t window;
  const int32_t* key_starts;
  float* weights;
  uint16_t* out;
  RangeInfo* info;
  float2* final_ml;
  float2* ml;
  float* o;
  float* scores;
  int64_t seq_units;  // units that `scores` holds per sequence
  int32_t used_ranges;  // ranges (by_cta: eights of them) that the longest lengths could fill
  int32_t range_step;   // by_cta: 8
  unsigned int* err;
};

// The visible tokens [lo, ctx) of a sequence; empty (0, 0) where there are none or the length is bad.
__device__ __forceinline__ int2 visible(const DecodeModParams& p, int b, bool report) {
  int ctx = p.context_lens[b];
  int lo = p.key_starts ? max(p.key_starts[b], 0) : 0;
  if (ctx < 0 || ctx > p.max_ctx || ctx > static_cast<int64_t>(p.bt_stride) * kBlockSize) {
    if (report) flag_error(p.err, PKV_DEVERR_BAD_SEQLEN);
    ctx = 0;
  }
  if (p.window > 0) lo = max(lo, ctx - p.window);
  return lo < ctx ? make_int2(lo, ctx) : make_int2(0, 0);
}
__device__ __forceinline__ int units_of(int2 v) {
  return v.y == 0 ? 0 : (v.y + kUnit - 1) / kUnit - v.x / kUnit;
}
__device__ __forceinline__ int64_t range_start(int r, int64_t units, int32_t ranges) {
  if (units < (1 << 20)) return static_cast<uint32_t>(r) * static_cast<uint32_t>(units) / static_cast<uint32_t>(ranges);
  return r * units / ranges;  // a 64-bit division takes some 0.3 us
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst_smem, const void* tmap, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst_smem),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&d)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&d)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <Elem E>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (E == Elem::kBF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void sts128_zero(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}

// Walks a worker's range: the sequence and the unit within it, and the block that holds it.
struct Walk {
  int b;          // sequence
  int2 seen;      // its visible tokens
  int unit;       // absolute unit (token / kUnit) of the sequence
  int last;       // the sequence's last unit
};

__device__ __forceinline__ void add_piece(float& M, float& L, float4& o, float2 ml, float4 x) {
  const float top = fmaxf(M, ml.x), use = top == -INFINITY ? 0.f : top;
  const float a = ex2_approx(M - use), b = ex2_approx(ml.x - use);
  M = top;
  L = L * a + ml.y * b;
  o.x = o.x * a + x.x * b;
  o.y = o.y * a + x.y * b;
  o.z = o.z * a + x.z * b;
  o.w = o.w * a + x.w * b;
}
template <Elem E>
__device__ __forceinline__ void write_joined(const DecodeModParams& p, int seq, int h, int lane, float M, float L, float4 o) {
  using Ops = ElemOps<E>;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t row = static_cast<int64_t>(seq) * p.hq + h;
  *(reinterpret_cast<uint2*>(p.out + row * kHeadDim) + lane) =
      make_uint2(Ops::pack(o.x * inv, o.y * inv), Ops::pack(o.z * inv, o.w * inv));
  if (p.weights && lane == 0) p.final_ml[row] = make_float2(M, inv);
}

// Which of a lane's 16 dims (2 i: 16 i + lane / 4, 2 i + 1: 8 more) hold +infinity (bits 0 to 15 of the result), -infinity
// (16 to 31) and NaN (32 to 47) among the values of tokens from..to - 1 of sequence b.
template <Elem E>
__device__ __noinline__ uint64_t odd_values(const DecodeModParams& p, int b, int hk, int from, int to) {
  constexpr uint32_t kInf = E == Elem::kBF16 ? 0x7f80u : 0x7c00u;
  const int lane = threadIdx.x & 31;
  uint32_t odd = 0;  // of dims 4 lane .. 4 lane + 3: bits 0 to 3, 4 to 7 and 8 to 11
  for (int t0 = from & ~15; t0 < to; t0 += 16) {
    int block = p.block_tables[static_cast<int64_t>(b) * p.bt_stride + t0 / kBlockSize];
    if (block < 0 || block >= p.num_blocks) block = 0;  // reported where it was fetched
    const int64_t row = (static_cast<int64_t>(block) * kBlockSize + t0 % kBlockSize) * p.hkv + hk;
    const uint16_t* rows = p.v + row * kHeadDim + 4 * lane;
    uint2 x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      x[j] = t0 + j >= from && t0 + j < to
                 ? *reinterpret_cast<const uint2*>(rows + static_cast<int64_t>(j) * p.hkv * kHeadDim) : make_uint2(0u, 0u);
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t e = ((d < 2 ? x[j].x : x[j].y) >> (16 * (d & 1))) & 0xffffu, size = e & 0x7fffu;
        if (size >= kInf) odd |= 1u << (d + (size > kInf ? 8 : (e >> 15 ? 4 : 0)));
      }
  }
  uint64_t mine = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int dim = 8 * i + lane / 4;
    const uint32_t there = __shfl_sync(0xffffffffu, odd, dim >> 2) >> (dim & 3);
    mine |= static_cast<uint64_t>(there & 1u) << i | static_cast<uint64_t>((there >> 4) & 1u) << (16 + i) |
            static_cast<uint64_t>((there >> 8) & 1u) << (32 + i);
  }
  return mine;
}

// NT: eights of query heads that a worker takes.
template <Elem E, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    decode_mod_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const DecodeModParams p) {
  using Ops = ElemOps<E>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  int64_t* scan = reinterpret_cast<int64_t*>(smem + kOffScan);  // units before each thread's sequences
  int64_t* warp_units = scan + kThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = sbase + warp * kStages * 2 * kUnitBytes;
  const uint32_t bars = sbase + kOffBars + warp * kStages * 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel may be set up beside this one
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
    mbar_fence_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }

  // ---- the units of all sequences, laid end to end ----
  const int B = p.num_seqs;
  const int per = (B + kThreads - 1) / kThreads;  // consecutive sequences per thread
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    const int n = b < B ? units_of(visible(p, b, blockIdx.x == 0)) : 0;
    mine += n;
    // sequences that see no key: zeros
    uint32_t empty = __ballot_sync(0xffffffffu, n == 0 && b < B && b % gridDim.x == blockIdx.x);
    for (; empty; empty &= empty - 1) {
      const int64_t row = (warp * 32 + __ffs(empty) - 1) * per + i;
      uint4* o = reinterpret_cast<uint4*>(p.out + row * p.hq * kHeadDim);
      for (int j = lane; j < p.hq * (kHeadDim / 8); j += 32) o[j] = make_uint4(0, 0, 0, 0);
    }
  }
  int64_t sum = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, sum, off);
    if (lane >= off) sum += y;
  }
  if (lane == 31) warp_units[warp] = sum;
  __syncthreads();
  int64_t before = 0, units = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_units[w];
    units += warp_units[w];
  }
  scan[tid] = before + sum - mine;
  __syncthreads();
  const int64_t fill = (units + kMinUnits - 1) / kMinUnits;
  const int ranges = static_cast<int>(fill < p.st.ranges ? fill : p.st.ranges);
  const int worker = static_cast<int>(blockIdx.x) * kWarps + warp;
  const int workers = static_cast<int>(gridDim.x) * kWarps;
  // A stream has all its ranges, or (more streams than workers) one range and a worker several streams.
  const bool split = p.st.ranges > 1, by_cta = p.st.by_cta != 0;
  const int cta_range = static_cast<int>(blockIdx.x) / p.st.count;  // by_cta: which eight ranges
  const int range = by_cta ? cta_range * kWarps + warp : (split ? worker / p.st.count : 0);
  Piece* pieces = reinterpret_cast<Piece*>(smem + kOffPieces);
  if (lane < 2) pieces[2 * warp + lane].seq = -1;
  __syncwarp();
  const bool idle = range >= ranges;
  if (idle && !by_cta) {
    if (split && lane == 0 && worker % p.st.count == 0 && range < p.used_ranges) p.info[range].seq = -1;
    return;
  }
  const int64_t start = idle ? 0 : range_start(range, units, ranges);
  const int64_t end = idle ? 0 : range_start(range + 1, units, ranges);

  // the sequence that holds unit `start`
  Walk begin{};
  int64_t begin_first = 0;  // first unit of begin.b
  if (!idle) {
    int at = 0;
#pragma unroll
    for (int j = 0; j < kThreads / 32; ++j) at += __popc(__ballot_sync(0xffffffffu, scan[j * 32 + lane] <= start));
    begin_first = scan[at - 1];
    begin.b = (at - 1) * per;
    while (true) {
      begin.seen = visible(p, begin.b, false);
      const int n = units_of(begin.seen);
      if (begin_first + n > start) break;
      begin_first += n;
      ++begin.b;
    }
    begin.last = (begin.seen.y - 1) / kUnit;
    begin.unit = begin.seen.x / kUnit + static_cast<int>(start - begin_first);
  }

  const int row16 = (lane & 7) + ((lane >> 3) & 1) * 8;  // ldmatrix: this lane's row of K
  const int rowv = (lane & 7) + (lane >> 4) * 8;         // and of V
  const int r = lane >> 2, c = lane & 3;                 // fragment row and column pair
  uint32_t phase = 0;                                    // bit i: parity of the next wait on stage i
  int stage = 0;
  bool ok = true;

  const int first_stream = by_cta ? static_cast<int>(blockIdx.x) % p.st.count : (split ? worker % p.st.count : worker);
  for (int stream = first_stream; !idle && stream < p.st.count && ok; stream += workers) {
    const int hk = stream / p.st.parts, part = stream - hk * p.st.parts;
    const int head0 = hk * p.st.group + part * p.st.per;
    const int heads = min(p.st.per, p.st.group - part * p.st.per);

    // ---- fetching, kStages units ahead ----
    Walk ahead = begin;
    int64_t to_fetch = end - start;
    int under_way = 0;                               // copies not waited for
    int block = -1, next_block = -1, block_at = -1;  // table entries; block_at: table place of `block`
    auto fetch = [&](int slot) {
      if (ahead.unit > ahead.last) {  // the next sequence with units
        do {
          ++ahead.b;
          ahead.seen = visible(p, ahead.b, false);
        } while (ahead.seen.y == 0);
        ahead.unit = ahead.seen.x / kUnit;
        ahead.last = (ahead.seen.y - 1) / kUnit;
        block_at = -1;
      }
      const int place = ahead.unit / (kBlockSize / kUnit);
      if (place != block_at) {
        const int32_t* table = p.block_tables + static_cast<int64_t>(ahead.b) * p.bt_stride;
        block = block_at >= 0 ? next_block : table[place];
        block_at = place;
        next_block = place < (ahead.seen.y - 1) / kBlockSize ? table[place + 1] : 0;
        if (block < 0 || block >= p.num_blocks) {
          if (lane == 0) flag_error(p.err, PKV_DEVERR_BAD_BLOCK);
          block = 0;
        }
      }
      if (lane == 0) {
        const int row = block * kBlockSize + (ahead.unit % (kBlockSize / kUnit)) * kUnit;
        const uint32_t bar = bars + 8 * slot, dst = ring + slot * 2 * kUnitBytes;
        mbar_arrive_expect_tx(bar, 2 * kUnitBytes);
        tma_load_4d(dst, &tm_k, 0, row, hk, 0, bar);
        tma_load_4d(dst + kUnitBytes, &tm_v, 0, row, hk, 0, bar);
      }
      ++ahead.unit;
      --to_fetch;
      ++under_way;
    };
    {
      int slot = stage;
      for (int i = 0; i < kStages && to_fetch > 0; ++i) {
        fetch(slot);
        slot = slot + 1 == kStages ? 0 : slot + 1;
      }
    }

    // A worker whose wait runs out leaves before it can say what goes on behind its range: nothing, then.
    const bool tells = !by_cta && stream == 0 && lane == 0;
    if (tells) p.info[range].seq = -1;
    Walk now = begin;
    int64_t first_unit = begin_first;  // of the sequence under way
    int64_t left = end - start;
    while (left > 0 && ok) {
      // ---- one sequence's units in this range ----
      const int n = static_cast<int>(min(left, static_cast<int64_t>(now.last - now.unit + 1)));
      const int seq_first = now.unit;
      // Q as the second operand: lane (r, c) holds head r, dims 16 i + 2 c, + 1 and + 8, + 9
      uint32_t qf[NT][8][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int h = 8 * t + r;
        const uint16_t* row = p.q + now.b * p.q_row_stride + static_cast<int64_t>(head0 + h) * kHeadDim + 2 * c;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            qf[t][i][j] = h < heads ? *reinterpret_cast<const uint32_t*>(row + 16 * i + 8 * j) : 0u;
      }
      float slope[NT][2], m[NT][2], l[NT][2], acc[NT][8][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int h = 8 * t + 2 * c + j;
          slope[t][j] = p.slopes && h < heads ? p.slopes[head0 + h] * kLog2e : 0.f;
          m[t][j] = -INFINITY;
          l[t][j] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[t][i][j] = 0.f;
      }

      for (int u = 0; u < n; ++u) {
        const int token0 = (seq_first + u) * kUnit;
        const uint32_t bar = bars + 8 * stage;
        const uint32_t ks = ring + stage * 2 * kUnitBytes, vs = ks + kUnitBytes;
        if (!__all_sync(0xffffffffu, mbar_wait(bar, (phase >> stage) & 1u, p.err))) {
          ok = false;
          break;
        }
        phase ^= 1u << stage;
        --under_way;
        const bool edge = token0 < now.seen.x || token0 + kUnit > now.seen.y;
        if (edge) {  // rows of V that are not visible may hold anything: 0 * NaN must not be added
          const int token = token0 + (lane >> 1);
          if (token < now.seen.x || token >= now.seen.y) {
            const uint32_t row = vs + (lane & 1) * (kUnitBytes / 2) + (lane >> 1) * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) sts128_zero(row + 16 * i);
          }
          fence_proxy_async_smem();  // before a later copy into the same place
          __syncwarp();
        }

        // S^T = K Q^T; two chains to halve the latency
        float s[NT][2][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 8; ++j) s[t][j >> 2][j & 3] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t a[4];
          const int chunk = 2 * i + (lane >> 4);
          ldmatrix_x4(ks + (chunk >> 3) * (kUnitBytes / 2) + row16 * 128 + (((chunk & 7) ^ (row16 & 7)) << 4), a);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816<E>(s[t][i & 1], a, qf[t][i][0], qf[t][i][1]);
        }

        // scores in log2 units; lane (r, c): tokens r, r + 8 of heads 2 c, 2 c + 1
        float z[NT][4];
        bool rise = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = s[t][0][j] + s[t][1][j];
            z[t][j] = p.cap_log2 > 0.f ? p.cap_log2 * tanhf(x * p.scale_by_cap) : x * p.scale_log2;
            const int token = token0 + r + (j >> 1) * 8;
            if (p.slopes) z[t][j] = fmaf(-slope[t][j & 1], static_cast<float>(now.seen.y - 1 - token), z[t][j]);
            if (edge && (token < now.seen.x || token >= now.seen.y)) z[t][j] = -INFINITY;
            rise = rise || z[t][j] > m[t][j & 1] + (8.f + kLift<E>);
          }
        if (p.weights) {
          float* to = p.scores + ((now.b * p.seq_units + (seq_first + u)) * p.st.count + stream) * (p.st.heads * kUnit);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int h = 8 * t + 2 * c + (j & 1);
              if (h < heads) to[h * kUnit + r + (j >> 1) * 8] = z[t][j];
            }
        }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float top = fmaxf(z[t][j], z[t][j + 2]);
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
              top = fmaxf(top - kLift<E>, m[t][j]);
              const float alpha = m[t][j] == -INFINITY ? 0.f : ex2_approx(m[t][j] - top);
              m[t][j] = top;
              l[t][j] *= alpha;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                acc[t][i][j] *= alpha;
                acc[t][i][j + 2] *= alpha;
              }
            }
        }
        // p, and what rounding it to 16 bits loses, as the second operand of the product with V
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            e[j] = ex2_approx(z[t][j] - (m[t][j & 1] == -INFINITY ? 0.f : m[t][j & 1]));
            l[t][j & 1] += e[j];
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t hi = Ops::pack(e[2 * j], e[2 * j + 1]);
            ph[t][j] = movmatrix(hi);
            pl[t][j] = movmatrix(Ops::pack(e[2 * j] - Ops::lo(hi), e[2 * j + 1] - Ops::hi(hi)));
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t a[4];
          const int chunk = 2 * i + ((lane >> 3) & 1);
          ldmatrix_x4_trans(vs + (chunk >> 3) * (kUnitBytes / 2) + rowv * 128 + (((chunk & 7) ^ (rowv & 7)) << 4), a);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16816<E>(acc[t][i], a, ph[t][0], ph[t][1]);
            mma16816<E>(acc[t][i], a, pl[t][0], pl[t][1]);
          }
        }
        __syncwarp();
        if (to_fetch > 0) fetch(stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
      }
      if (!ok) break;

      // A value that is infinite makes NaN with the second part of p, which may be 0 or of the other sign. Where a sum is
      // NaN the values are looked through: those of one infinity alone make that.
      {
        float spoilt = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) spoilt = fmaf(acc[t][i][j], 0.f, spoilt);
        if (__any_sync(0xffffffffu, isnan(spoilt))) {
          const uint64_t odd = odd_values<E>(p, now.b, hk, max(seq_first * kUnit, now.seen.x),
                                             min((seq_first + n) * kUnit, now.seen.y));
          const uint32_t nan = static_cast<uint32_t>(odd >> 32), up = static_cast<uint32_t>(odd) & 0xffffu;
          const uint32_t down = static_cast<uint32_t>(odd) >> 16;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t bit = 1u << (2 * i + (j >> 1));
                if (isnan(acc[t][i][j]) && !(nan & bit) && ((up ^ down) & bit))
                  acc[t][i][j] = up & bit ? INFINITY : -INFINITY;
              }
        }
      }

      // ---- the end of a sequence, or of the range inside one ----
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], off);
      const bool begins = first_unit >= start;              // this range holds its first unit
      const bool ends = now.unit + n > now.last;            // and its last
      if (begins && ends) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float inv0 = l[t][0] == 0.f ? 0.f : 1.f / l[t][0], inv1 = l[t][1] == 0.f ? 0.f : 1.f / l[t][1];
          uint16_t* row = p.out + (static_cast<int64_t>(now.b) * p.hq + head0 + 8 * t + r) * kHeadDim + 2 * c;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t x = movmatrix(Ops::pack(acc[t][i][0] * inv0, acc[t][i][1] * inv1));
            const uint32_t y = movmatrix(Ops::pack(acc[t][i][2] * inv0, acc[t][i][3] * inv1));
            if (8 * t + r < heads) {
              *reinterpret_cast<uint32_t*>(row + 16 * i) = x;
              *reinterpret_cast<uint32_t*>(row + 16 * i + 8) = y;
            }
          }
          if (p.weights && r == 0) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int h = 8 * t + 2 * c + j;
              if (h < heads)
                p.final_ml[static_cast<int64_t>(now.b) * p.hq + head0 + h] = make_float2(m[t][j], j ? inv1 : inv0);
            }
          }
        }
      } else {
        const int place = first_unit <= start ? 0 : 1;
        const int64_t slot = ((static_cast<int64_t>(range) * p.st.count + stream) * 2 + place) * p.st.heads;
        float* o_to = p.o + slot * kHeadDim;
        float2* ml_to = p.ml + slot;
        if (by_cta) {
          if (left == n) {  // no copies under way
            o_to = reinterpret_cast<float*>(smem + warp * kStages * 2 * kUnitBytes);
            ml_to = reinterpret_cast<float2*>(o_to + p.st.heads * kHeadDim);
          }
          if (lane == 0) {
            Piece& piece = pieces[2 * warp + place];
            piece.seq = now.b;
            piece.ends = ends;
            piece.first_unit = first_unit;
            piece.end_unit = first_unit + (now.last - now.seen.x / kUnit + 1);
            piece.ml = ml_to;
            piece.o = o_to;
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int h = 8 * t + 2 * c + j;
            if (h < heads) {
              float* o = o_to + h * kHeadDim + r;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                o[16 * i] = acc[t][i][j];
                o[16 * i + 8] = acc[t][i][j + 2];
              }
              if (r == 0) ml_to[h] = make_float2(m[t][j], l[t][j]);
            }
          }
      }
      left -= n;
      if (left == 0) {
        if (tells) {
          const int64_t last_unit = first_unit + (now.last - now.seen.x / kUnit);
          RangeInfo info;
          info.seq = begins && !ends ? now.b : -1;
          info.last = static_cast<int>(((last_unit + 1) * ranges - 1) / units);
          info.place = first_unit <= start ? 0 : 1;
          info.pad = 0;
          *reinterpret_cast<int4*>(p.info + range) = *reinterpret_cast<const int4*>(&info);
        }
      } else {
        first_unit += now.last - now.seen.x / kUnit + 1;
        do {
          ++now.b;
          now.seen = visible(p, now.b, false);
        } while (now.seen.y == 0);
        now.unit = now.seen.x / kUnit;
        now.last = (now.seen.y - 1) / kUnit;
      }
    }
    if (!ok) {  // leave no copy in flight
      for (int i = 0; i < under_way; ++i)
        mbar_wait(bars + 8 * ((stage + i) % kStages), (phase >> ((stage + i) % kStages)) & 1u, p.err);
    }
  }
  if (!by_cta) return;

  // ---- the CTA's pieces, joined in order: pieces of one sequence lie side by side ----
  __syncthreads();
  const int stream = first_stream, hk = stream / p.st.parts, part = stream - hk * p.st.parts;
  const int head0 = hk * p.st.group + part * p.st.per;
  const int heads = min(p.st.per, p.st.group - part * p.st.per);
  const int64_t cta_start = cta_range * kWarps < ranges ? range_start(cta_range * kWarps, units, ranges) : 0;
  RangeInfo goes_on;
  goes_on.seq = -1;
  goes_on.last = goes_on.place = goes_on.pad = 0;
  for (int i = 0, group = 0; i < kPieces; ++group) {
    const Piece first = pieces[i];
    if (first.seq < 0) {
      ++i;
      --group;
      continue;
    }
    int n = i + 1;       // one behind the sequence's last piece here
    bool ends = first.ends != 0;
    for (int k = i + 1; k < kPieces; ++k) {
      if (pieces[k].seq < 0) continue;
      if (pieces[k].seq != first.seq) break;
      ends = pieces[k].ends != 0;
      n = k + 1;
    }
    const bool begins = first.first_unit >= cta_start;
    const int place = first.first_unit <= cta_start ? 0 : 1;
    for (int h = (warp - group) & (kWarps - 1); h < heads; h += kWarps) {
      float M = -INFINITY, L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = i; k < n; ++k) {
        if (pieces[k].seq < 0) continue;
        const float2 ml = pieces[k].ml[h];
        const float4 x = *(reinterpret_cast<const float4*>(pieces[k].o + h * kHeadDim) + lane);
        add_piece(M, L, o, ml, x);
      }
      if (begins && ends) {
        write_joined<E>(p, first.seq, head0 + h, lane, M, L, o);
      } else {
        const int64_t slot = ((static_cast<int64_t>(cta_range) * kWarps * p.st.count + stream) * 2 + place) * p.st.heads + h;
        *(reinterpret_cast<float4*>(p.o + slot * kHeadDim) + lane) = o;
        if (lane == 0) p.ml[slot] = make_float2(M, L);
      }
    }
    if (begins && !ends) {
      goes_on.seq = first.seq;
      goes_on.last = static_cast<int>((first.end_unit * ranges - 1) / units) / kWarps;
      goes_on.place = place;
    }
    i = n;
  }
  if (stream == 0 && tid == 0 && cta_range < p.used_ranges)
    *reinterpret_cast<int4*>(p.info + cta_range) = *reinterpret_cast<const int4*>(&goes_on);
}

// Partial results r = first, first + step, ... up to last of one query head, joined: (max, sum) and four dims to a lane.
__device__ __forceinline__ void join(const DecodeModParams& p, int range, int place, int stream, int in_part, int first,
                                     int last, int step, int lane, float& M, float& L, float4& o) {
  constexpr int kAhead = 10;
  M = -INFINITY;
  L = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r0 = first; r0 <= last; r0 += step * kAhead) {
    float2 ml[kAhead];
    float4 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = min(r0 + i * step, last);
      const int64_t slot =
          ((static_cast<int64_t>(r) * p.range_step * p.st.count + stream) * 2 + (r == range ? place : 0)) * p.st.heads + in_part;
      ml[i] = p.ml[slot];
      x[i] = *(reinterpret_cast<const float4*>(p.o + slot * kHeadDim) + lane);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (r0 + i * step > last) break;
      add_piece(M, L, o, ml[i], x[i]);
    }
  }
}

// Whether {seq, last, place} can be what a range's worker has left: workspaces need no initialisation, so nothing else is
// followed, not even where a wait that ran out has kept a worker from writing it.
__device__ __forceinline__ bool fits(const DecodeModParams& p, int range, int seq, int last, int place) {
  return seq >= 0 && seq < p.num_seqs && last >= range && last < p.used_ranges && place >= 0 && place <= 1;
}

// A block joins what one query head of the sequences left that begin in its kMergeWarps ranges and go on behind them:
// a warp each those of few pieces, all warps together those of many.
template <Elem E>
__global__ void __launch_bounds__(kMergeWarps * 32) decode_mod_merge_kernel(const DecodeModParams p) {
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  __shared__ int s_info[kMergeWarps][3];
  __shared__ float4 s_o[kMergeWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = static_cast<int>(blockIdx.y);
  const int hk = h / p.st.group, in_group = h - hk * p.st.group, part = in_group / p.st.per;
  const int stream = hk * p.st.parts + part, in_part = in_group - part * p.st.per;
  const int first = static_cast<int>(blockIdx.x) * kMergeWarps;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float M, L;
  float4 o;
  const int ranges = p.used_ranges;
  if (first + warp < ranges) {
    int4 info = *reinterpret_cast<const int4*>(p.info + first + warp);  // {seq, last, place}
    if (!fits(p, first + warp, info.x, info.y, info.z)) info.x = -1;
    s_info[warp][0] = info.x;
    s_info[warp][1] = info.y;
    s_info[warp][2] = info.z;
    if (info.x >= 0 && info.y - (first + warp) < kMergeWarps) {
      join(p, first + warp, info.z, stream, in_part, first + warp, info.y, 1, lane, M, L, o);
      write_joined<E>(p, info.x, h, lane, M, L, o);
    }
  }
  __syncthreads();
  for (int i = 0; i < min(kMergeWarps, ranges - first); ++i) {
    const int range = first + i, seq = s_info[i][0], last = s_info[i][1];
    if (seq < 0 || last - range < kMergeWarps) continue;
    join(p, range, s_info[i][2], stream, in_part, range + warp, last, kMergeWarps, lane, M, L, o);
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = L;
    }
    s_o[warp][lane] = o;
    __syncthreads();
    if (warp == 0) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, s_m[w]);
      const float use = top == -INFINITY ? 0.f : top;
      L = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float a = ex2_approx(s_m[w] - use);
        const float4 y = s_o[w][lane];
        L += s_l[w] * a;
        o.x += y.x * a;
        o.y += y.y * a;
        o.z += y.z * a;
        o.w += y.w * a;
      }
      write_joined<E>(p, seq, h, lane, top, L, o);
    }
    __syncthreads();
  }
}

// weights[t] += the share of t among its sequence's scores, summed over the query heads of a kv head; the newest token's
// starts from 0. One block per (256-token block of a sequence); a thread takes four tokens of every fourth kv head.
__global__ void __launch_bounds__(kBlockSize) decode_mod_weights_kernel(const DecodeModParams p) {
  const int b = static_cast<int>(blockIdx.y), place = static_cast<int>(blockIdx.x);
  const int quad = static_cast<int>(threadIdx.x) & 63, token = place * kBlockSize + 4 * quad;
  const int2 seen = visible(p, b, false);
  const int ctx = p.context_lens[b];
  const bool good = ctx > 0 && ctx <= p.max_ctx && ctx <= static_cast<int64_t>(p.bt_stride) * kBlockSize;
  if (!good || place > (ctx - 1) / kBlockSize || (place + 1) * kBlockSize <= min(seen.x, ctx - 1)) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int block = p.block_tables[static_cast<int64_t>(b) * p.bt_stride + place];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (block < 0 || block >= p.num_blocks) return;  // reported where it was fetched
  bool shown[4], any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    shown[i] = token + i >= seen.x && token + i < seen.y;
    any = any || shown[i] || token + i == ctx - 1;
  }
  if (!any) return;
  const int newest = ctx - 1 - token;  // 0..3: one of these
  float4* w = reinterpret_cast<float4*>(p.weights + static_cast<int64_t>(block) * p.hkv * kBlockSize) + quad;
  const int z_stride = p.st.heads * (kUnit / 4);  // float4 per stream
  const float4* z0 = reinterpret_cast<const float4*>(p.scores) +
                     (b * p.seq_units + token / kUnit) * p.st.count * z_stride + (quad & (kUnit / 4 - 1));
  const float2* ml0 = p.final_ml + static_cast<int64_t>(b) * p.hq;
  constexpr int kHeads = 2;  // kv heads whose loads are on the way together
  for (int h0 = static_cast<int>(threadIdx.x) >> 6; h0 < p.hkv; h0 += 4 * kHeads) {
    float4 old[kHeads];
    float share[kHeads][4];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int hk = min(h0 + 4 * i, p.hkv - 1);
      old[i] = w[static_cast<int64_t>(hk) * (kBlockSize / 4)];
#pragma unroll
      for (int j = 0; j < 4; ++j) share[i][j] = 0.f;
    }
#pragma unroll 2
    for (int g = 0; g < p.st.group; ++g) {
      const int part = g / p.st.per, in_part = g - part * p.st.per;
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int hk = min(h0 + 4 * i, p.hkv - 1);
        const float4 z = z0[(hk * p.st.parts + part) * z_stride + in_part * (kUnit / 4)];
        const float2 ml = ml0[hk * p.st.group + g];
        const float zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          share[i][j] += shown[j] && ml.y != 0.f ? ex2_approx(zs[j] - ml.x) * ml.y : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (h0 + 4 * i >= p.hkv) break;
      auto added = [&](int j, float before) { return newest == j ? share[i][j] : (shown[j] ? before + share[i][j] : before); };
      w[static_cast<int64_t>(h0 + 4 * i) * (kBlockSize / 4)] =
          make_float4(added(0, old[i].x), added(1, old[i].y), added(2, old[i].z), added(3, old[i].w));
    }
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

// A cache as [half of the dims][head][slot][64 dims], so that one copy brings both 128-byte halves of kUnit rows.
bool encode_cache(CUtensorMap* tm, const void* base, int64_t slots, int heads, Elem elem) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(slots), static_cast<cuuint64_t>(heads), 2};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(heads) * kHeadDim * 2, kHeadDim * 2, kHeadDim};
  const cuuint32_t box[4] = {64, kUnit, 1, 2};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType dt = elem == Elem::kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(tm, dt, 4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch whose blocks may be set up while the kernel before it ends (each waits for that one's results itself).
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

template <Elem E, int NT>
cudaError_t launch_typed(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeModParams& p, int ctas,
                         cudaStream_t stream) {
  static std::atomic<bool> attr_done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  const bool known = dev >= 0 && dev < 64;
  if (!known || !attr_done[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(decode_mod_kernel<E, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    if (known) attr_done[dev].store(true, std::memory_order_release);
  }
  decode_mod_kernel<E, NT><<<ctas, kThreads, kSmemBytes, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

size_t decode_mod_workspace_bytes(int32_t num_seqs, int32_t hq, int32_t hkv, int32_t max_ctx, bool weights) {
  return layout_of(streams_of(hq, hkv, num_seqs, max_ctx), num_seqs, hq, max_ctx, weights).total;
}

cudaError_t launch_decode_mod(const DecodeModArgs& a, unsigned int* err, cudaStream_t stream, Elem elem) {
  const Streams st = streams_of(a.hq, a.hkv, a.num_seqs, a.max_ctx);
  const bool weights = a.weights != nullptr;
  const Layout lay = layout_of(st, a.num_seqs, a.hq, a.max_ctx, weights);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  DecodeModParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_row_stride = a.q_row_stride;
  p.v = static_cast<const uint16_t*>(a.v_cache);
  p.block_tables = a.block_tables;
  p.bt_stride = a.bt_stride;
  p.num_blocks = a.num_blocks;
  p.context_lens = a.context_lens;
  p.num_seqs = a.num_seqs;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.max_ctx = a.max_ctx;
  p.st = st;
  p.scale_log2 = a.scale * kLog2e;
  const float cap = a.softcap < kNoCap ? a.softcap : 0.f;
  p.cap_log2 = cap * kLog2e;
  p.scale_by_cap = cap > 0.f ? fminf(a.scale / cap, FLT_MAX) : 0.f;  // not infinity: a score of 0 stays 0
  p.slopes = a.slopes;
  p.window = a.window;
  p.key_starts = a.key_starts;
  p.weights = a.weights;
  p.out = static_cast<uint16_t*>(a.out);
  p.info = reinterpret_cast<RangeInfo*>(ws + lay.info);
  p.final_ml = reinterpret_cast<float2*>(ws + lay.final_ml);
  p.ml = reinterpret_cast<float2*>(ws + lay.ml);
  p.o = reinterpret_cast<float*>(ws + lay.o);
  p.scores = reinterpret_cast<float*>(ws + lay.scores);
  p.seq_units = (static_cast<int64_t>(a.max_ctx) + kUnit - 1) / kUnit;
  p.err = err;
  CUtensorMap tk, tv;
  const int64_t slots = static_cast<int64_t>(a.num_blocks) * kBlockSize;
  if (!encode_cache(&tk, a.k_cache, slots, a.hkv, elem) || !encode_cache(&tv, a.v_cache, slots, a.hkv, elem))
    return cudaErrorInvalidValue;
  // no more workers than the longest lengths could keep busy
  const int64_t fill = (p.seq_units * a.num_seqs + kMinUnits - 1) / kMinUnits;
  const int32_t used = static_cast<int32_t>(fill < st.ranges ? fill : st.ranges);
  p.range_step = st.by_cta ? kWarps : 1;
  p.used_ranges = (used + p.range_step - 1) / p.range_step;
  const int64_t want = st.by_cta ? static_cast<int64_t>(p.used_ranges) * st.count
                                 : (fill * st.count + kWarps - 1) / kWarps;
  const int ctas = static_cast<int>(want < 1 ? 1 : (want < kCtas ? want : kCtas));
  const bool f16 = elem == Elem::kF16;
  cudaError_t e;
  if (st.per == 8)
    e = f16 ? launch_typed<Elem::kF16, 1>(tk, tv, p, ctas, stream) : launch_typed<Elem::kBF16, 1>(tk, tv, p, ctas, stream);
  else
    e = f16 ? launch_typed<Elem::kF16, 2>(tk, tv, p, ctas, stream) : launch_typed<Elem::kBF16, 2>(tk, tv, p, ctas, stream);
  if (e != cudaSuccess) return e;
  if (st.ranges > 1 && p.used_ranges > 0) {
    const dim3 grid(static_cast<unsigned>((p.used_ranges + kMergeWarps - 1) / kMergeWarps), static_cast<unsigned>(a.hq));
    e = launch_behind(f16 ? decode_mod_merge_kernel<Elem::kF16> : decode_mod_merge_kernel<Elem::kBF16>, grid,
                      kMergeWarps * 32, stream, p);
    if (e != cudaSuccess) return e;
  }
  if (weights && a.max_ctx > 0) {
    const dim3 grid(static_cast<unsigned>((a.max_ctx + kBlockSize - 1) / kBlockSize), static_cast<unsigned>(a.num_seqs));
    e = launch_behind(decode_mod_weights_kernel, grid, kBlockSize, stream, p);
  }
  return e;
}

}  // namespace pkv

namespace {

constexpr int32_t kMaxHeads = 8192;
constexpr int32_t kMaxBlocks = (1 << 23) - 1;  // slots are 32-bit coordinates of the copies

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool heads_fit(int32_t hq, int32_t hkv) { return hkv > 0 && hq > 0 && hq <= kMaxHeads && hq % hkv == 0; }

int decode_mod_common(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                      int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                      const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                      int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale,
                      float softcap, const float* slopes, int32_t window, const int32_t* key_starts, float* weights,
                      void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream, pkv::Elem elem) {
  if (head_dim != pkv::kHeadDim || block_size != pkv::kBlockSize || !heads_fit(num_heads, num_kv_heads))
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs < 0 || num_seqs > 65535 || num_blocks < 0 || num_blocks > kMaxBlocks || block_table_stride < 0 ||
      max_context_len < 0 || max_context_len > (1 << 24) || window < 0)
    return PKV_ERR_BAD_SIZE;
  if (num_seqs == 0) return PKV_OK;
  if (!(softmax_scale > 0.f) || std::isinf(softmax_scale) || !(softcap >= 0.f) || std::isinf(softcap))
    return PKV_ERR_BAD_SIZE;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out) return PKV_ERR_NULL_POINTER;
  if (num_blocks == 0) return PKV_ERR_BAD_SIZE;
  if (q_row_stride < static_cast<int64_t>(num_heads) * head_dim) return PKV_ERR_BAD_STRIDE;
  if (!aligned(q, 16) || q_row_stride % 8 != 0 || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(out, 16) || !aligned(slopes, 4) || !aligned(key_starts, 4) || !aligned(weights, 16))
    return PKV_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < pkv::decode_mod_workspace_bytes(num_seqs, num_heads, num_kv_heads,
                                                                      max_context_len, weights != nullptr))
    return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return PKV_ERR_ALIGNMENT;
  unsigned int* err = nullptr;
  const int st = pkv::device_error_word(&err);
  if (st != PKV_OK) return st;
  pkv::DecodeModArgs a{};
  a.q = q;
  a.q_row_stride = q_row_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_blocks = num_blocks;
  a.block_tables = block_tables;
  a.bt_stride = block_table_stride;
  a.context_lens = context_lens;
  a.num_seqs = num_seqs;
  a.hq = num_heads;
  a.hkv = num_kv_heads;
  a.max_ctx = max_context_len;
  a.scale = softmax_scale;
  a.softcap = softcap;
  a.slopes = slopes;
  a.window = window;
  a.key_starts = key_starts;
  a.weights = weights;
  a.out = out;
  a.workspace = workspace;
  if (pkv::launch_decode_mod(a, err, stream, elem) == cudaSuccess) return PKV_OK;
  (void)cudaGetLastError();
  return PKV_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t pkv_decode_mod_workspace_bytes(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                      int32_t max_context_len, int32_t weights) {
  if (num_seqs <= 0 || num_seqs > 65535 || max_context_len < 0 || max_context_len > (1 << 24) ||
      !heads_fit(num_heads, num_kv_heads))
    return 0;
  return pkv::decode_mod_workspace_bytes(num_seqs, num_heads, num_kv_heads, max_context_len, weights != 0);
}

// The bf16 and fp16 entry points share one body; only the elements' type differs.

int pkv_decode_mod(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache, int32_t num_blocks,
                   const int32_t* block_tables, int32_t block_table_stride, const int32_t* context_lens,
                   int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                   int32_t max_context_len, float softmax_scale, float softcap, const float* slopes, int32_t window,
                   const int32_t* key_starts, float* weights, void* out, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream) {
  return decode_mod_common(q, q_row_stride, k_cache, v_cache, num_blocks, block_tables, block_table_stride,
                           context_lens, num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                           softmax_scale, softcap, slopes, window, key_starts, weights, out, workspace,
                           workspace_bytes, stream, pkv::Elem::kBF16);
}

int pkv_decode_mod_f16(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                       int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                       const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                       int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale,
                       float softcap, const float* slopes, int32_t window, const int32_t* key_starts, float* weights,
                       void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return decode_mod_common(q, q_row_stride, k_cache, v_cache, num_blocks, block_tables, block_table_stride,
                           context_lens, num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                           softmax_scale, softcap, slopes, window, key_starts, weights, out, workspace,
                           workspace_bytes, stream, pkv::Elem::kF16);
}

}  // extern "C"
