// rope.cu -- rotary positions of queries and keys, alone or fused with the store of the step's K and V rows.
//
// Pair i of a head (elements i and i + r/2 in the half layout, 2i and 2i + 1 in the interleaved one, i < r/2) turns by
// the angle position * f_i:   a' = a cos - b sin,   b' = b cos + a sin   (both times a factor that some scalings use).
// Elements from r on are copied.
//
// The angle: f_i is held as a 64-bit fixed-point number of full turns per position (2^-64 of a turn), so the low 64 bits
// of position * f_i are the exact fraction of a turn, at any position and with no table of cosines to read. Its upper 32
// bits as a signed number, rounded to fp32 (at most 2^-26 of a turn), go to sincospif: the angle is off by less than
// 2^-23 rad, an eighth of what rounding the result to fp16 loses. fp32 products of position and frequency, instead,
// are off by 2^-24 of the whole angle: 0.008 rad at position 131072.
//
// HBM bound: q, k (and v) are read once and written once. A block takes a few tokens: its threads compute the tokens'
// r/2 cosines and sines once, for all heads, into shared memory while their first rows are on the way; then a thread
// moves 32 bytes at a time (eight pairs). The fused form writes turned keys and values to their slots, which saves the
// keys' way through memory (2 x 2 KB of the 16 KB a token of 16 heads on 8 costs in two calls) and a launch. Measured:
// 15 k tokens of 16 heads on 8 29.1 us, with the store 37.0 (0.79 and 0.83 of a plain copy's rate) with the L2 full of other
// data, 25.9 and 35.1 again and again on the same rows, of which a part is in the L2 then; 5 tokens take 2.0 us, 256 with
// the store 2.6, on the device; their calls from Python 11.6 and 14.9.
#include <cmath>
#include <type_traits>

#include "pkv_common.cuh"

namespace pkv {

struct RopeArgs {
  const void* q;
  int64_t q_stride;
  const void* k;
  int64_t k_stride;
  const void* v;  // with slots only
  int64_t v_stride;
  void* q_out;
  int64_t q_out_stride;
  void* k_out;  // rows, or the cache where slots are given
  int64_t k_out_stride;
  void* v_out;
  const int64_t* positions;
  const int64_t* freqs;
  const int32_t* slots;
  int64_t num_slots;
  int32_t num_tokens, hq, hkv, d, rot;
  float magnitude;
};

namespace {

constexpr int kThreads = 256;
// Tokens per block at most, and 32-byte pieces that a thread has on the way. 15 k tokens of 16 heads on 8, half of each
// fp16 head turned | all of it, bf16, with the store: 8 and 3 25.9 | 35.1 us (6.0 | 5.9 TB/s), 4 and 4 27.6 | 37.0, 1 and
// 4 48.7 | 65.4, 16 and 3 29.5 | 36.6.
constexpr int kMaxTokens = 8;
constexpr int kBatch = 3;

struct RopeParams {
  const uint16_t* src[3];  // q, k, v
  int64_t src_stride[3];
  uint16_t* dst[3];
  int64_t dst_stride[3];
  const int64_t* positions;
  const int64_t* freqs;
  const int32_t* slots;
  int64_t num_slots;
  int32_t num_tokens, hq, hkv, d, half;
  int32_t tokens;  // per block
  float magnitude;
  unsigned int* err;
};

__device__ __forceinline__ uint4 ld_row16(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// cos and sin of the angle, times the magnitude
__device__ __forceinline__ float2 cos_sin(int64_t position, int64_t freq, float magnitude) {
  const uint64_t turn = static_cast<uint64_t>(position) * static_cast<uint64_t>(freq);
  const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

// Cosines and sines of the block's tokens, and their slots (-1: not stored).
template <bool kStore>
__device__ __forceinline__ void block_angles(const RopeParams& p, int first, int n, float* cosines, float* sines,
                                             int64_t* slots) {
  for (int i = threadIdx.x; i < n * p.half; i += kThreads) {
    const int t = i / p.half;
    const float2 cs = cos_sin(p.positions[first + t], p.freqs[i - t * p.half], p.magnitude);
    cosines[i] = cs.x;
    sines[i] = cs.y;
  }
  if (kStore && threadIdx.x < n) {
    int64_t slot = p.slots[first + threadIdx.x];
    if (slot < 0 || slot >= p.num_slots) {
      if (slot != -1) flag_error(p.err, PKV_DEVERR_BAD_SLOT);
      slot = -1;
    }
    slots[threadIdx.x] = slot;
  }
}

// 32-bit words of two elements: x holds firsts, y seconds of a pair (half layout)
template <Elem E>
__device__ __forceinline__ void turn_word(uint32_t& x, uint32_t& y, float c0, float s0, float c1, float s1) {
  using Ops = ElemOps<E>;
  const float a0 = Ops::lo(x), a1 = Ops::hi(x), b0 = Ops::lo(y), b1 = Ops::hi(y);
  x = Ops::pack(fmaf(a0, c0, -b0 * s0), fmaf(a1, c1, -b1 * s1));
  y = Ops::pack(fmaf(b0, c0, a0 * s0), fmaf(b1, c1, a1 * s1));
}
// a word holds one pair (interleaved layout)
template <Elem E>
__device__ __forceinline__ void turn_pair(uint32_t& x, float c, float s) {
  using Ops = ElemOps<E>;
  const float a = Ops::lo(x), b = Ops::hi(x);
  x = Ops::pack(fmaf(a, c, -b * s), fmaf(b, c, a * s));
}

// Rows are q's heads, then k's, then (kStore) v's. A thread keeps its place in the head, a piece of eight pairs or, past
// the turned part and in v, of 16 elements, and goes over the block's (token, row) pairs. Needs 16-byte alignment
// throughout, d and the turned part in multiples of 16.
template <Elem E, bool kInterleaved, bool kStore>
__global__ void __launch_bounds__(kThreads, 4) rope_v16_kernel(const RopeParams p) {
  extern __shared__ __align__(16) float angles[];  // [tokens][half] cosines, then sines
  __shared__ int64_t slots[kMaxTokens];
  const int first = static_cast<int>(blockIdx.x) * p.tokens;
  const int n = min(p.tokens, p.num_tokens - first);
  float* cosines = angles;
  float* sines = angles + p.tokens * p.half;

  const int pieces = p.d >> 4;
  const int rows = p.hq + p.hkv + (kStore ? p.hkv : 0);
  const int step = kThreads / pieces;  // rows a block moves at once
  const int piece = static_cast<int>(threadIdx.x) % pieces;
  const bool turned = piece < (p.half >> 3);
  const int off0 = !kInterleaved && turned ? 8 * piece : 16 * piece;
  const int off1 = !kInterleaved && turned ? p.half + 8 * piece : 16 * piece + 8;
  int at = static_cast<int>(threadIdx.x) / pieces;
  if (at >= step) at = n * rows;  // threads left over
  // the next row to load
  int t = at / rows, row = at - t * rows;

  uint4 x[kBatch], y[kBatch];
  uint16_t* to[kBatch];  // where the row goes but for the slot
  int8_t what[kBatch];   // -1: nothing, else 2 * (token of the block) + (1: a row of the cache); turned rows have bit 4
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      what[i] = -1;
      if (t < n) {
        const int part = row < p.hq ? 0 : (row < p.hq + p.hkv ? 1 : 2);
        const int head = row - (part > 0 ? p.hq : 0) - (part > 1 ? p.hkv : 0);
        const uint16_t* s = p.src[part] + (first + t) * p.src_stride[part] + head * p.d;
        x[i] = ld_row16(s + off0 + (kStore && part == 2 ? 16 * piece - off0 : 0));
        y[i] = ld_row16(s + off1 + (kStore && part == 2 ? 16 * piece + 8 - off1 : 0));
        const bool cached = kStore && part > 0;
        to[i] = p.dst[part] + (cached ? 0 : (first + t) * p.dst_stride[part]) + head * p.d;
        what[i] = static_cast<int8_t>((part == 2 ? 0 : 16) | (2 * t) | (cached ? 1 : 0));
        row += step;
        while (row >= rows) {
          row -= rows;
          ++t;
        }
      }
    }
  };
  load();
  block_angles<kStore>(p, first, n, cosines, sines, slots);
  __syncthreads();
  while (what[0] >= 0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (what[i] < 0) continue;
      const int token = (what[i] >> 1) & 7;
      uint16_t* d0 = to[i];
      bool write = true;
      int o0 = off0, o1 = off1;
      if (kStore && (what[i] & 1)) {
        const int64_t slot = slots[token];
        write = slot >= 0;
        d0 += slot * p.dst_stride[1];
      }
      if (kStore && !(what[i] & 16)) {
        o0 = 16 * piece;
        o1 = o0 + 8;
      } else if (turned) {
        const float4* cp = reinterpret_cast<const float4*>(cosines + token * p.half + 8 * piece);
        const float4* sp = reinterpret_cast<const float4*>(sines + token * p.half + 8 * piece);
        const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
        if (kInterleaved) {
          turn_pair<E>(x[i].x, c0.x, s0.x);
          turn_pair<E>(x[i].y, c0.y, s0.y);
          turn_pair<E>(x[i].z, c0.z, s0.z);
          turn_pair<E>(x[i].w, c0.w, s0.w);
          turn_pair<E>(y[i].x, c1.x, s1.x);
          turn_pair<E>(y[i].y, c1.y, s1.y);
          turn_pair<E>(y[i].z, c1.z, s1.z);
          turn_pair<E>(y[i].w, c1.w, s1.w);
        } else {
          turn_word<E>(x[i].x, y[i].x, c0.x, s0.x, c0.y, s0.y);
          turn_word<E>(x[i].y, y[i].y, c0.z, s0.z, c0.w, s0.w);
          turn_word<E>(x[i].z, y[i].z, c1.x, s1.x, c1.y, s1.y);
          turn_word<E>(x[i].w, y[i].w, c1.z, s1.z, c1.w, s1.w);
        }
      }
      if (write) {
        *reinterpret_cast<uint4*>(d0 + o0) = x[i];
        *reinterpret_cast<uint4*>(d0 + o1) = y[i];
      }
    }
    load();
  }
}

// Any turned part: a thread moves 16-byte pieces, and finds the partners of the turned elements in one in what the others
// have read (in the half layout they lie anywhere in the row; in one piece if a half is a whole number of them). Since
// rows may be turned in place, a batch of whole rows is read before any of it is written. Needs 16-byte alignment
// throughout and d in multiples of 8. 5.5 k tokens of 32 heads on 8, 6 of 128 dims, with the store: 49 us (interleaved 31);
// partners fetched from the rows once more 60, a pair at a time 183; one piece a thread at once 47 (33), four 63 (34).
constexpr int kBatch8 = 2;
template <Elem E, bool kInterleaved, bool kStore>
__global__ void __launch_bounds__(kThreads, 5) rope_v8_kernel(const RopeParams p) {
  using Ops = ElemOps<E>;
  extern __shared__ __align__(16) float angles[];
  __shared__ uint4 read[2][kBatch8][kThreads];  // what the threads have read, in turns: the pieces of a row lie side by side
  __shared__ int64_t slots[kMaxTokens];
  const int first = static_cast<int>(blockIdx.x) * p.tokens;
  const int n = min(p.tokens, p.num_tokens - first);
  float* cosines = angles;
  float* sines = angles + p.tokens * p.half;
  block_angles<kStore>(p, first, n, cosines, sines, slots);
  __syncthreads();
  const int pieces = p.d >> 3;
  const int rows = p.hq + p.hkv + (kStore ? p.hkv : 0);
  const int step = kThreads / pieces;  // rows a block moves at once
  const int e0 = 8 * (static_cast<int>(threadIdx.x) % pieces);
  const int at = static_cast<int>(threadIdx.x) / pieces;
  const int end = at < step ? n * rows : 0;  // (threads left over)
  const bool whole = p.half % 8 == 0;
  int turn = 0;
  for (int r0 = 0; r0 < n * rows; r0 += step * kBatch8) {
    uint4 x[kBatch8];
    uint16_t* to[kBatch8];
    int token[kBatch8];  // of the block, where this piece is turned; else -1
#pragma unroll
    for (int i = 0; i < kBatch8; ++i) {
      const int r = r0 + i * step + at;
      to[i] = nullptr;
      token[i] = -1;
      if (r >= end) continue;
      const int t = r / rows, row = r - t * rows;
      const int part = row < p.hq ? 0 : (row < p.hq + p.hkv ? 1 : 2);
      const int head = row - (part > 0 ? p.hq : 0) - (part > 1 ? p.hkv : 0);
      int64_t line = first + t;
      if (kStore && part > 0) {
        line = slots[t];
        if (line < 0) continue;
      }
      const uint16_t* s = p.src[part] + (first + t) * p.src_stride[part] + head * p.d;
      to[i] = p.dst[part] + line * p.dst_stride[part] + head * p.d + e0;
      x[i] = ld_row16(s + e0);
      if (!kInterleaved) read[turn][i][threadIdx.x] = x[i];
      if (part < 2 && e0 < 2 * p.half) token[i] = t;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBatch8; ++i) {
      if (token[i] < 0) continue;
      const uint16_t* s = reinterpret_cast<const uint16_t*>(&read[turn][i][at * pieces]);  // the row
      uint32_t* w = &x[i].x;
      const float* cs = cosines + token[i] * p.half;
      const float* sn = sines + token[i] * p.half;
      if (kInterleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pair = (e0 >> 1) + j;
          if (pair < p.half) turn_pair<E>(w[j], cs[pair], sn[pair]);
        }
      } else if (whole) {
        const bool second = e0 >= p.half;
        const int pair = second ? e0 - p.half : e0;
        uint4 y = *reinterpret_cast<const uint4*>(s + (second ? pair : pair + p.half));
        uint32_t* v = &y.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (second)
            turn_word<E>(v[j], w[j], cs[pair + 2 * j], sn[pair + 2 * j], cs[pair + 2 * j + 1], sn[pair + 2 * j + 1]);
          else
            turn_word<E>(w[j], v[j], cs[pair + 2 * j], sn[pair + 2 * j], cs[pair + 2 * j + 1], sn[pair + 2 * j + 1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float r2[2] = {Ops::lo(w[j]), Ops::hi(w[j])};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int e = e0 + 2 * j + h;
            if (e >= 2 * p.half) continue;
            const bool second = e >= p.half;
            const int pair = second ? e - p.half : e;
            const float y = Ops::lo(s[second ? pair : pair + p.half]);
            r2[h] = second ? fmaf(r2[h], cs[pair], y * sn[pair]) : fmaf(r2[h], cs[pair], -y * sn[pair]);
          }
          w[j] = Ops::pack(r2[0], r2[1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch8; ++i)
      if (to[i]) *reinterpret_cast<uint4*>(to[i]) = x[i];
    turn ^= 1;
  }
}

// Any sizes and alignment: one pair, or one element that is copied, at a time.
template <Elem E, bool kInterleaved, bool kStore>
__global__ void __launch_bounds__(kThreads) rope_u16_kernel(const RopeParams p) {
  using Ops = ElemOps<E>;
  extern __shared__ __align__(16) float angles[];
  __shared__ int64_t slots[kMaxTokens];
  const int first = static_cast<int>(blockIdx.x) * p.tokens;
  const int n = min(p.tokens, p.num_tokens - first);
  float* cosines = angles;
  float* sines = angles + p.tokens * p.half;
  block_angles<kStore>(p, first, n, cosines, sines, slots);
  __syncthreads();
  const int rows = p.hq + p.hkv + (kStore ? p.hkv : 0);
  const int units = p.d - p.half;  // pairs, then copied elements
  for (int t = 0; t < n; ++t) {
    for (int64_t i = threadIdx.x; i < static_cast<int64_t>(rows) * p.d; i += kThreads) {
      const int row = static_cast<int>(i / p.d), e = static_cast<int>(i - static_cast<int64_t>(row) * p.d);
      const int part = row < p.hq ? 0 : (row < p.hq + p.hkv ? 1 : 2);
      const int head = row - (part > 0 ? p.hq : 0) - (part > 1 ? p.hkv : 0);
      if (part < 2 && e >= units) continue;
      const uint16_t* s = p.src[part] + (first + t) * p.src_stride[part] + static_cast<int64_t>(head) * p.d;
      int64_t to = first + t;
      if (kStore && part > 0) {
        to = slots[t];
        if (to < 0) continue;
      }
      uint16_t* d = p.dst[part] + to * p.dst_stride[part] + static_cast<int64_t>(head) * p.d;
      if (part == 2) {
        d[e] = s[e];
      } else if (e >= p.half) {
        d[e + p.half] = s[e + p.half];
      } else {
        const int a = kInterleaved ? 2 * e : e, b = kInterleaved ? 2 * e + 1 : e + p.half;
        const float c = cosines[t * p.half + e], sn = sines[t * p.half + e];
        const float xa = Ops::lo(s[a]), xb = Ops::lo(s[b]);
        const uint32_t r = Ops::pack(fmaf(xa, c, -xb * sn), fmaf(xb, c, xa * sn));
        d[a] = static_cast<uint16_t>(r & 0xffffu);
        d[b] = static_cast<uint16_t>(r >> 16);
      }
    }
  }
}

bool vec16(const void* p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; }

template <Elem E, bool kInterleaved, bool kStore>
void launch_typed(const RopeParams& p, bool vector, unsigned blocks, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(p.tokens) * p.half * 8;
  if (vector && p.d % 16 == 0 && p.half % 8 == 0)
    rope_v16_kernel<E, kInterleaved, kStore><<<blocks, kThreads, smem, stream>>>(p);
  else if (vector)
    rope_v8_kernel<E, kInterleaved, kStore><<<blocks, kThreads, smem, stream>>>(p);
  else
    rope_u16_kernel<E, kInterleaved, kStore><<<blocks, kThreads, smem, stream>>>(p);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool interleaved, unsigned int* err, cudaStream_t stream, Elem elem) {
  const bool store = a.slots != nullptr;
  RopeParams p{};
  p.src[0] = static_cast<const uint16_t*>(a.q);
  p.src[1] = static_cast<const uint16_t*>(a.k);
  p.src[2] = static_cast<const uint16_t*>(a.v);
  p.src_stride[0] = a.q_stride;
  p.src_stride[1] = a.k_stride;
  p.src_stride[2] = a.v_stride;
  p.dst[0] = static_cast<uint16_t*>(a.q_out);
  p.dst[1] = static_cast<uint16_t*>(a.k_out);
  p.dst[2] = static_cast<uint16_t*>(a.v_out);
  p.dst_stride[0] = a.q_out_stride;
  p.dst_stride[1] = p.dst_stride[2] = a.k_out_stride;
  p.positions = a.positions;
  p.freqs = a.freqs;
  p.slots = a.slots;
  p.num_slots = a.num_slots;
  p.num_tokens = a.num_tokens;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.d = a.d;
  p.half = a.rot / 2;
  p.magnitude = a.magnitude;
  p.err = err;
  // Several tokens to a block spread the wait for the angles over more rows; with few tokens every SM should have some.
  p.tokens = 1;
  while (p.tokens < kMaxTokens && a.num_tokens >= 2 * p.tokens * 4 * 152) p.tokens *= 2;
  bool vector = a.d % 8 == 0 && a.d <= 8 * kThreads;
  if (a.hq > 0) vector = vector && vec16(a.q, a.q_stride) && vec16(a.q_out, a.q_out_stride);
  if (a.hkv > 0) vector = vector && vec16(a.k, a.k_stride) && vec16(a.k_out, a.k_out_stride);
  if (a.hkv > 0 && store) vector = vector && vec16(a.v, a.v_stride) && vec16(a.v_out, a.k_out_stride);
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(a.num_tokens) + p.tokens - 1) / p.tokens);
  const auto go = [&](auto e) {
    constexpr Elem E = decltype(e)::value;
    if (interleaved)
      store ? launch_typed<E, true, true>(p, vector, blocks, stream)
            : launch_typed<E, true, false>(p, vector, blocks, stream);
    else
      store ? launch_typed<E, false, true>(p, vector, blocks, stream)
            : launch_typed<E, false, false>(p, vector, blocks, stream);
  };
  if (elem == Elem::kF16)
    go(std::integral_constant<Elem, Elem::kF16>{});
  else
    go(std::integral_constant<Elem, Elem::kBF16>{});
  return cudaGetLastError();
}

// Frequencies in 2^-64 turns per position; false for arguments that give none.
bool rope_frequencies(int32_t rot, double theta, int32_t scaling, double factor, double original, double a, double b,
                      int64_t* out, float* magnitude) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  *magnitude = 1.f;
  if (scaling == PKV_ROPE_NTK && rot > 2) theta *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
  double low = 0, high = 0;
  if (scaling == PKV_ROPE_YARN) {  // the pairs that turn a and b times over the original length
    *magnitude = static_cast<float>(0.1 * std::log(factor) + 1.0);
    low = std::floor(rot * std::log(original / (a * kTwoPi)) / (2 * std::log(theta)));
    high = std::ceil(rot * std::log(original / (b * kTwoPi)) / (2 * std::log(theta)));
    low = low > 0 ? low : 0;
    high = high < rot - 1 ? high : rot - 1;
  }
  for (int32_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot);
    if (scaling == PKV_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == PKV_ROPE_BANDS) {
      double keep = (original * f / kTwoPi - a) / (b - a);
      keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
      f = f / factor * (1 - keep) + f * keep;
    } else if (scaling == PKV_ROPE_YARN) {
      const double span = high - low > 0.001 ? high - low : 0.001;
      double ramp = (i - low) / span;
      ramp = ramp < 0 ? 0 : (ramp > 1 ? 1 : ramp);
      f = f / factor * ramp + f * (1 - ramp);
    }
    const double turns = f / kTwoPi;
    if (!(turns >= 0 && turns < 0.5)) return false;
    out[i] = static_cast<int64_t>(turns * 0x1p64);
  }
  return true;
}

}  // namespace pkv

namespace {

constexpr int32_t kMaxHeadDim = 1024;
constexpr int32_t kMaxHeads = 8192;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int rope_common(pkv::RopeArgs a, const void* const* needed, int num_needed, int32_t interleaved, cudaStream_t stream,
                pkv::Elem elem) {
  if (a.d < 1 || a.d > kMaxHeadDim || a.rot < 2 || a.rot % 2 != 0 || a.rot > a.d || a.hq < 0 || a.hq > kMaxHeads ||
      a.hkv < 0 || a.hkv > kMaxHeads)
    return PKV_ERR_UNSUPPORTED;
  if (a.num_tokens < 0 || a.num_slots < 0) return PKV_ERR_BAD_SIZE;
  if (a.num_tokens == 0 || (a.hq == 0 && a.hkv == 0)) return PKV_OK;
  if (!std::isfinite(a.magnitude)) return PKV_ERR_BAD_SIZE;
  if (!a.positions || !a.freqs) return PKV_ERR_NULL_POINTER;
  const int64_t q_row = static_cast<int64_t>(a.hq) * a.d, k_row = static_cast<int64_t>(a.hkv) * a.d;
  if (a.hq > 0 && (!a.q || !a.q_out)) return PKV_ERR_NULL_POINTER;
  if (a.hkv > 0)
    for (int i = 0; i < num_needed; ++i)
      if (!needed[i]) return PKV_ERR_NULL_POINTER;
  if (a.hq > 0 && (a.q_stride < q_row || a.q_out_stride < q_row)) return PKV_ERR_BAD_STRIDE;
  if (a.hkv > 0 && (a.k_stride < k_row || a.k_out_stride < k_row || (a.v && a.v_stride < k_row)))
    return PKV_ERR_BAD_STRIDE;
  for (const void* p : {a.q, a.k, a.v, static_cast<const void*>(a.q_out), static_cast<const void*>(a.k_out),
                        static_cast<const void*>(a.v_out)})
    if (!aligned(p, 2)) return PKV_ERR_ALIGNMENT;
  if (!aligned(a.positions, 8) || !aligned(a.freqs, 8) || !aligned(a.slots, 4)) return PKV_ERR_ALIGNMENT;
  unsigned int* err = nullptr;
  const int st = pkv::device_error_word(&err);
  if (st != PKV_OK) return st;
  if (pkv::launch_rope(a, interleaved != 0, err, stream, elem) == cudaSuccess) return PKV_OK;
  (void)cudaGetLastError();
  return PKV_ERR_CUDA;
}

int rope_alone(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const int64_t* positions,
               const int64_t* freqs, int32_t rotary_dim, float magnitude, int32_t interleaved, int32_t num_tokens,
               int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, void* q_out, int64_t q_out_row_stride,
               void* k_out, int64_t k_out_row_stride, cudaStream_t stream, pkv::Elem elem) {
  pkv::RopeArgs a{};
  a.q = q;
  a.q_stride = q_row_stride;
  a.k = k;
  a.k_stride = k_row_stride;
  a.q_out = q_out;
  a.q_out_stride = q_out_row_stride;
  a.k_out = k_out;
  a.k_out_stride = k_out_row_stride;
  a.positions = positions;
  a.freqs = freqs;
  a.num_tokens = num_tokens;
  a.hq = num_heads;
  a.hkv = num_kv_heads;
  a.d = head_dim;
  a.rot = rotary_dim;
  a.magnitude = magnitude;
  const void* needed[] = {k, k_out};
  return rope_common(a, needed, 2, interleaved, stream, elem);
}

int rope_store(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
               int64_t v_row_stride, const int64_t* positions, const int64_t* freqs, int32_t rotary_dim,
               float magnitude, int32_t interleaved, const int32_t* slot_mapping, int32_t num_tokens,
               int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int64_t num_slots, void* q_out,
               int64_t q_out_row_stride, void* k_cache, void* v_cache, cudaStream_t stream, pkv::Elem elem) {
  pkv::RopeArgs a{};
  a.q = q;
  a.q_stride = q_row_stride;
  a.k = k;
  a.k_stride = k_row_stride;
  a.v = v;
  a.v_stride = v_row_stride;
  a.q_out = q_out;
  a.q_out_stride = q_out_row_stride;
  a.k_out = k_cache;
  a.k_out_stride = static_cast<int64_t>(num_kv_heads) * head_dim;
  a.v_out = v_cache;
  a.positions = positions;
  a.freqs = freqs;
  a.slots = num_kv_heads > 0 ? slot_mapping : nullptr;  // no keys: the turned queries alone
  a.num_slots = num_slots;
  a.num_tokens = num_tokens;
  a.hq = num_heads;
  a.hkv = num_kv_heads;
  a.d = head_dim;
  a.rot = rotary_dim;
  a.magnitude = magnitude;
  const void* needed[] = {k, v, k_cache, v_cache, slot_mapping};
  return rope_common(a, needed, 5, interleaved, stream, elem);
}

}  // namespace

extern "C" {

int pkv_rope_frequencies(int32_t rotary_dim, double theta, int32_t scaling, double factor,
                         double original_max_position, double a, double b, int64_t* h_freqs, float* h_magnitude) {
  if (!h_freqs || !h_magnitude) return PKV_ERR_NULL_POINTER;
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > kMaxHeadDim || scaling < PKV_ROPE_NONE ||
      scaling > PKV_ROPE_YARN)
    return PKV_ERR_UNSUPPORTED;
  if (!std::isfinite(theta) || !(theta > 1)) return PKV_ERR_BAD_SIZE;
  if (scaling != PKV_ROPE_NONE && (!std::isfinite(factor) || !(factor >= 1))) return PKV_ERR_BAD_SIZE;
  if (scaling == PKV_ROPE_BANDS || scaling == PKV_ROPE_YARN) {
    if (!std::isfinite(original_max_position) || !(original_max_position >= 1) || !std::isfinite(a) || !std::isfinite(b))
      return PKV_ERR_BAD_SIZE;
    if (scaling == PKV_ROPE_BANDS ? !(a < b) : !(a > b && b > 0)) return PKV_ERR_BAD_SIZE;
  }
  return pkv::rope_frequencies(rotary_dim, theta, scaling, factor, original_max_position, a, b, h_freqs, h_magnitude)
             ? PKV_OK
             : PKV_ERR_BAD_SIZE;
}

// The bf16 and fp16 entry points share one body each; only the elements' type differs.

int pkv_rope(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const int64_t* positions,
             const int64_t* freqs, int32_t rotary_dim, float magnitude, int32_t interleaved, int32_t num_tokens,
             int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, void* q_out, int64_t q_out_row_stride,
             void* k_out, int64_t k_out_row_stride, cudaStream_t stream) {
  return rope_alone(q, q_row_stride, k, k_row_stride, positions, freqs, rotary_dim, magnitude, interleaved, num_tokens,
                    num_heads, num_kv_heads, head_dim, q_out, q_out_row_stride, k_out, k_out_row_stride, stream,
                    pkv::Elem::kBF16);
}

int pkv_rope_f16(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const int64_t* positions,
                 const int64_t* freqs, int32_t rotary_dim, float magnitude, int32_t interleaved, int32_t num_tokens,
                 int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, void* q_out, int64_t q_out_row_stride,
                 void* k_out, int64_t k_out_row_stride, cudaStream_t stream) {
  return rope_alone(q, q_row_stride, k, k_row_stride, positions, freqs, rotary_dim, magnitude, interleaved, num_tokens,
                    num_heads, num_kv_heads, head_dim, q_out, q_out_row_stride, k_out, k_out_row_stride, stream,
                    pkv::Elem::kF16);
}

int pkv_rope_store_kvcache(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                           int64_t v_row_stride, const int64_t* positions, const int64_t* freqs, int32_t rotary_dim,
                           float magnitude, int32_t interleaved, const int32_t* slot_mapping, int32_t num_tokens,
                           int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int64_t num_slots, void* q_out,
                           int64_t q_out_row_stride, void* k_cache, void* v_cache, cudaStream_t stream) {
  return rope_store(q, q_row_stride, k, k_row_stride, v, v_row_stride, positions, freqs, rotary_dim, magnitude,
                    interleaved, slot_mapping, num_tokens, num_heads, num_kv_heads, head_dim, num_slots, q_out,
                    q_out_row_stride, k_cache, v_cache, stream, pkv::Elem::kBF16);
}

int pkv_rope_store_kvcache_f16(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                               int64_t v_row_stride, const int64_t* positions, const int64_t* freqs,
                               int32_t rotary_dim, float magnitude, int32_t interleaved, const int32_t* slot_mapping,
                               int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                               int64_t num_slots, void* q_out, int64_t q_out_row_stride, void* k_cache, void* v_cache,
                               cudaStream_t stream) {
  return rope_store(q, q_row_stride, k, k_row_stride, v, v_row_stride, positions, freqs, rotary_dim, magnitude,
                    interleaved, slot_mapping, num_tokens, num_heads, num_kv_heads, head_dim, num_slots, q_out,
                    q_out_row_stride, k_cache, v_cache, stream, pkv::Elem::kF16);
}

}  // extern "C"
