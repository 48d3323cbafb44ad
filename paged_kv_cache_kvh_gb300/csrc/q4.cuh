// q4.cuh -- the 4-bit paged KV cache: format, quantiser and reader (sm_103a).
//
// One (token, kv head) row of K or of V is 128 dims in 4 groups of 32. A group
// keeps a scale s = fp16((max - min) / 15) and a minimum z = fp16(min), a dim
// keeps the code c = clamp(round_half_even((x - z) / s), 0, 15) (0 where s is
// 0), and stands for s * c + z. |x| above 65504 counts as 65504; a group with
// a NaN or an infinity has s = z = NaN, so it reads back as NaN.
//
// Cache layout, uint8 [num_blocks, num_kv_heads, 16, 1280]: a 256-token block
// is 16 tiles of 16 tokens per head, a tile is 16 x 64 bytes of codes and then
// 16 x 4 x (s, z) in fp16. The tokens of one head are contiguous, so any run
// of whole tiles of a (block, head) is one bulk copy. Within a code row:
//   K: the 32-bit word at byte 16 t + 4 j holds dims 32 j + 8 t + p, p = 0..7,
//      code p in bits 4p..4p+3.
//   V: the 8-byte chunk r sits at chunk place r ^ (4 if token & 4 else 0); its
//      16-bit field j holds dims 32 j + 4 r + p, p = 0..3.
// Both orders are those of the decode kernel's tensor-core operands: a K row's
// 16 bytes at 16 t are one lane's share of a fragment, and a 16-byte half chunk
// pair of V, transposed by the load, is four dims of every group. The swap of the
// V halves spreads 8 tokens' 16-byte pieces over more banks.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

constexpr int kQ4Tile = 16;                                   // tokens per tile
constexpr int kQ4CodeBytes = 64;                              // one row's codes
constexpr int kQ4ParamBytes = 16;                             // one row's 4 x (s, z)
constexpr int kQ4TileBytes = kQ4Tile * (kQ4CodeBytes + kQ4ParamBytes);  // 1280
constexpr int kQ4TileParams = kQ4Tile * kQ4CodeBytes;         // parameters' offset in a tile
constexpr int kQ4RecordBytes = kBlockSize / kQ4Tile * kQ4TileBytes;     // one (block, head): 20480
constexpr float kF16Max = 65504.f;

__device__ __forceinline__ float2 h2_to_f2(uint32_t packed) {
  return __half22float2(*reinterpret_cast<const __half2*>(&packed));
}

__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Packed pair max / min that keep a NaN of either operand.
template <Elem E>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  if (E == Elem::kBF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <Elem E>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  if (E == Elem::kBF16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The scale, the minimum and what the codes are computed with, of a group whose
// packed (pairwise) maximum and minimum are given.
struct Q4Group {
  uint32_t param;  // s in the low half, z in the high half
  float s, z;
  float rs;        // 1 / s, off by 2^-22 of it at most; 0 where s is 0
  bool plain;      // no quotient leaves [-0.5, 15.5], so none needs clamping
  bool finite;
};
template <Elem E>
__device__ __forceinline__ Q4Group q4_group(uint32_t mx2, uint32_t mn2) {
  using Ops = ElemOps<E>;
  mx2 = max2_nan<E>(mx2, __byte_perm(mx2, mx2, 0x1032));
  mn2 = min2_nan<E>(mn2, __byte_perm(mn2, mn2, 0x1032));
  const float mx = Ops::lo(mx2), mn = Ops::lo(mn2);
  Q4Group g;
  g.finite = fabsf(mx) < INFINITY && fabsf(mn) < INFINITY;  // false for NaN too
  const float hi = fminf(fmaxf(mx, -kF16Max), kF16Max), lo = fminf(fmaxf(mn, -kF16Max), kF16Max);
  const __half hs = __float2half_rn(__fdiv_rn(hi - lo, 15.f)), hz = __float2half_rn(lo);
  g.param = g.finite ? static_cast<uint32_t>(__half_as_ushort(hs)) | (static_cast<uint32_t>(__half_as_ushort(hz)) << 16)
                     : 0x7fff7fffu;
  g.s = __half2float(hs);
  g.z = __half2float(hz);
  g.rs = g.s > 0.f ? __fdividef(1.f, g.s) : 0.f;
  // A normal s is off by 2^-11 of itself, and z (exact in fp16 but below 2^-14,
  // where it is off by 2^-25) by 2^-11 s at most: quotients stay below 15.02.
  g.plain = g.finite && g.s >= 6.103515625e-5f && mx <= kF16Max && mn >= -kF16Max;
  return g;
}

// Codes of 8 elements, element p in bits 4p..4p+3. They are those of the
// definition exactly, also next to a border between two codes: the fp32 quotient
// is off by less than 15.5 * 2^-21 < 2^-17, so only elements whose quotient lies
// within 2^-16 of a border are decided again, from the sign of
// x - z - (k + 1/2) s. There the fp32 difference t = x - z cancels against
// (k + 1/2) s (16 bits) without rounding, and what t itself was rounded by is
// added back.
template <Elem E>
__device__ __forceinline__ uint32_t q4_codes(const uint4 raw, const Q4Group& g) {
  using Ops = ElemOps<E>;
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  constexpr float kNear = 0.5f - 1.52587890625e-5f;
  const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
  const uint64_t nz2 = f32x2_pack(-g.z, -g.z), rs2 = f32x2_pack(g.rs, g.rs);
  const uint64_t round2 = f32x2_pack(kRound, kRound), minus2 = f32x2_pack(-1.f, -1.f);
  float far = 0.f;
  uint32_t v[8];  // the rounded quotients as floats 1.5 * 2^23 + code
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t y = f32x2_mul(f32x2_add(f32x2_pack(Ops::lo(in[i]), Ops::hi(in[i])), nz2), rs2);
    const uint64_t r = f32x2_add(y, round2);
    float d0, d1, r0, r1;
    f32x2_unpack(f32x2_add(y, f32x2_fma(r, minus2, round2)), d0, d1);  // y - k, k = r - 1.5 * 2^23
    f32x2_unpack(r, r0, r1);
    far = fmax3(far, fabsf(d0), fabsf(d1));
    v[2 * i] = __float_as_uint(r0);
    v[2 * i + 1] = __float_as_uint(r1);
  }
  if (!(g.plain && far <= kNear)) {
    // (bf16 rows meet exact ties often enough for some lane of a warp to come
    // here in every fifth call)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = (i & 1) ? Ops::hi(in[i / 2]) : Ops::lo(in[i / 2]);
      const float t = x - g.z;
      float y = t * g.rs;
      if (!g.plain) y = fminf(fmaxf(y, 0.f), 15.f);
      const float r = y + kRound, k = r - kRound;
      const float d = y - k;
      v[i] = __float_as_uint(r);
      if (fabsf(d) > kNear) {
        const float lower = d > 0.f ? k : k - 1.f;
        const float b = t - x;
        const float lost = (x - (t - b)) + (-g.z - b);  // x - z == t + lost
        const float side = fmaf(-(lower + 0.5f), g.s, t) + lost;
        const uint32_t lo = __float_as_uint(lower + kRound);
        v[i] = lo + ((side > 0.f || (side == 0.f && (lo & 1u) != 0u)) ? 1u : 0u);
      }
      if (!g.finite) v[i] = 0u;
    }
  }
  // halves: codes 0..3 and 4..7; a code is the low 16 bits of v
  uint32_t w = __byte_perm(v[0], v[4], 0x5410);
#pragma unroll
  for (int i = 1; i < 4; ++i) w += __byte_perm(v[i], v[i + 4], 0x5410) << (4 * i);
  return w;
}

// Quantises 8 consecutive dims per lane; the 4 lanes of an aligned lane quad
// hold one group of 32 (all 32 lanes call this).
template <Elem E>
__device__ __forceinline__ uint32_t quantise8(const uint4 raw, uint32_t& param) {
  uint32_t mx2 = max2_nan<E>(max2_nan<E>(raw.x, raw.y), max2_nan<E>(raw.z, raw.w));
  uint32_t mn2 = min2_nan<E>(min2_nan<E>(raw.x, raw.y), min2_nan<E>(raw.z, raw.w));
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) {
    mx2 = max2_nan<E>(mx2, __shfl_xor_sync(0xffffffffu, mx2, off));
    mn2 = min2_nan<E>(mn2, __shfl_xor_sync(0xffffffffu, mn2, off));
  }
  const Q4Group g = q4_group<E>(mx2, mn2);
  param = g.param;
  return q4_codes<E>(raw, g);
}

// The same of 16 dims per lane, two lanes to a group: dims 8u.. (raw0) and
// 16 + 8u.. (raw1) of the group for lane u of an aligned pair.
template <Elem E>
__device__ __forceinline__ void quantise16(const uint4 raw0, const uint4 raw1, uint32_t& param, uint32_t& codes0,
                                           uint32_t& codes1) {
  uint32_t mx2 = max2_nan<E>(max2_nan<E>(max2_nan<E>(raw0.x, raw0.y), max2_nan<E>(raw0.z, raw0.w)),
                             max2_nan<E>(max2_nan<E>(raw1.x, raw1.y), max2_nan<E>(raw1.z, raw1.w)));
  uint32_t mn2 = min2_nan<E>(min2_nan<E>(min2_nan<E>(raw0.x, raw0.y), min2_nan<E>(raw0.z, raw0.w)),
                             min2_nan<E>(min2_nan<E>(raw1.x, raw1.y), min2_nan<E>(raw1.z, raw1.w)));
  mx2 = max2_nan<E>(mx2, __shfl_xor_sync(0xffffffffu, mx2, 1));
  mn2 = min2_nan<E>(mn2, __shfl_xor_sync(0xffffffffu, mn2, 1));
  const Q4Group g = q4_group<E>(mx2, mn2);
  param = g.param;
  codes0 = q4_codes<E>(raw0, g);
  codes1 = q4_codes<E>(raw1, g);
}

// The V word of lane (j, t) of a row's 16 lanes (lane 4 j + t): chunk
// 2 t + (j & 1), fields j & ~1 and j | 1, from every lane's own 8 dims 8 (4 j + t)...
__device__ __forceinline__ uint32_t v_exchange(uint32_t own, int j) {
  const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 4);
  return (j & 1) ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
}

// The same where 8 lanes share a row, lane 2 j + u holding t = u (own0) and
// t = u + 2 (own1): chunks 2 u + (j & 1) and 2 u + 4 + (j & 1). The exchange is
// its own inverse, so it also turns such words back into dims.
__device__ __forceinline__ void v_exchange2(uint32_t& own0, uint32_t& own1, int j) {
  const uint32_t send = (j & 1) ? __byte_perm(own0, own1, 0x5410) : __byte_perm(own0, own1, 0x7632);
  const uint32_t other = __shfl_xor_sync(0xffffffffu, send, 2);
  if (j & 1) {
    own0 = __byte_perm(other, own0, 0x7610);
    own1 = __byte_perm(other, own1, 0x7632);
  } else {
    own0 = __byte_perm(own0, other, 0x5410);
    own1 = __byte_perm(own1, other, 0x7610);
  }
}

// Byte offsets within a tile, for lane (j, t) of token `tok` of the tile.
__device__ __forceinline__ int q4_k_word(int tok, int j, int t) { return tok * kQ4CodeBytes + 16 * t + 4 * j; }
__device__ __forceinline__ int q4_v_word(int tok, int j, int t) {
  return tok * kQ4CodeBytes + ((2 * t + (j & 1)) ^ (tok & 4)) * 8 + (j >> 1) * 4;
}
__device__ __forceinline__ int q4_param(int tok, int j) { return kQ4TileParams + tok * kQ4ParamBytes + 4 * j; }

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(mask), "r"(bits));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// 8 codes -> 8 values s * c + z of the element type (dim p from bits 4p..4p+3).
//
// fp16: one fma.f16x2 per pair, so each value is s * c + z rounded once;
// saturated, since z + 15 s may pass 65504 by half a step of s. A nibble
// becomes a half by or-ing it into 1024, where it adds c (or 16 c).
//
// bf16: s * c + z in fp32, then rounded to bf16. kScaled values are 2^-64 times
// those (exactly, in bf16): the nibbles, and-ed out in place, are then used as
// they stand, as the fp32 subnormals c * 2^(4p - 149), with s * 2^(85 - 4p) as
// the factor (s < 2^16). Unscaled, that factor would overflow, so there a nibble
// is or-ed into 2^23 first and 2^23 taken off again.
template <Elem E, bool kScaled = false>
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, uint32_t param) {
  using Ops = ElemOps<E>;
  if constexpr (E == Elem::kF16) {
    const uint32_t s2 = __byte_perm(param, param, 0x1010), z2 = __byte_perm(param, param, 0x3232);
    const uint32_t high = codes >> 8;
    uint32_t v[4];  // dims (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? codes : high;
      const uint32_t n = (i & 1) ? hfma2(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd400d400u)   // / 16 - 64
                                 : hfma2(and_or(w, 0x000f000fu, 0x64006400u), 0x3c003c00u, 0xe400e400u);  // - 1024
      v[i] = min2_nan<E>(hfma2(n, s2, z2), 0x7bff7bffu);
    }
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                      __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
  } else {
    const float2 sz = h2_to_f2(param);
    const uint32_t high = codes >> 16;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // dims 2i, 2i + 1 and 2i + 4, 2i + 5
      const uint32_t m0 = 0xfu << (8 * i), m1 = 0xf0u << (8 * i);
      uint64_t lo, hi, f2, z2;
      if (kScaled) {
        // 2^(85 - 4p) of p = 2i and 2i + 1; 2^-64
        f2 = f32x2_pack(sz.x * __uint_as_float((127u + 85u - 8u * i) << 23),
                        sz.x * __uint_as_float((127u + 81u - 8u * i) << 23));
        const float z = sz.y * __uint_as_float((127u - 64u) << 23);
        z2 = f32x2_pack(z, z);
        lo = f32x2_pack(__uint_as_float(codes & m0), __uint_as_float(codes & m1));
        hi = f32x2_pack(__uint_as_float(high & m0), __uint_as_float(high & m1));
      } else {
        f2 = f32x2_pack(sz.x * __uint_as_float((127u - 8u * i) << 23), sz.x * __uint_as_float((123u - 8u * i) << 23));
        z2 = f32x2_pack(sz.y, sz.y);
        const uint64_t off2 = f32x2_pack(-8388608.f, -8388608.f);
        lo = f32x2_add(f32x2_pack(__uint_as_float(and_or(codes, m0, 0x4b000000u)),
                                  __uint_as_float(and_or(codes, m1, 0x4b000000u))), off2);
        hi = f32x2_add(f32x2_pack(__uint_as_float(and_or(high, m0, 0x4b000000u)),
                                  __uint_as_float(and_or(high, m1, 0x4b000000u))), off2);
      }
      float a, b;
      f32x2_unpack(f32x2_fma(lo, f2, z2), a, b);
      w[i] = Ops::pack(a, b);
      f32x2_unpack(f32x2_fma(hi, f2, z2), a, b);
      w[2 + i] = Ops::pack(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace pkv
