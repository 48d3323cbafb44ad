// q4_store.cu -- writing rows into the 4-bit paged cache and reading them back.
//
// pkv_store_kvcache_q4: token i's K and V rows, quantised, go to slot
// slot_mapping[i]; pkv_load_kvcache_q4 is its inverse, a gather of slots into
// 16-bit rows. The format and the quantiser are in q4.cuh.
//
// Both move (512 + 160) bytes per (token, kv head) and are bound by HBM, the
// store nearly as much by the instructions of the quantiser. Eight lanes share a
// row, lane 2 j + u holding 16 of group j's 32 dims, in two 16-byte pieces
// chosen so that each load or store of a warp covers whole 32-byte sectors; what
// a group costs once (its scale) is then spread over twice the elements that
// sixteen lanes to a row would give it. A 256-thread block takes 32 consecutive
// tokens of one kv head: where the slots are consecutive (a prompt) it covers two
// whole 1280-byte tiles of the cache. Heads vary fastest over the grid, so the
// blocks that share the tokens' rows run together.
#include "q4.cuh"

namespace pkv {

namespace {

constexpr int kRowsPerBlock = 32;
constexpr int kThreads = kRowsPerBlock * 8;

struct Q4RowsParams {
  const uint16_t* k;  // rows in (store); strides in elements
  const uint16_t* v;
  int64_t k_stride;
  int64_t v_stride;
  uint16_t* k_out;  // rows out (load), contiguous heads
  uint16_t* v_out;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int32_t* slot_mapping;
  int64_t num_slots;
  int32_t num_tokens;
  int32_t hkv;
  int32_t blocks_per_z;
  unsigned int* err;
};

__device__ __forceinline__ uint4 ld_rows_v4(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// The same 8 elements one at a time, for rows that are not 16-byte aligned.
__device__ __forceinline__ uint4 ld_rows_u16(const uint16_t* p) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = static_cast<uint32_t>(p[2 * i]) | (static_cast<uint32_t>(p[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The slot of this thread's row, or -1 where there is nothing to do.
__device__ __forceinline__ int64_t row_slot(const Q4RowsParams& p, int64_t token, bool report) {
  if (token >= p.num_tokens) return -1;
  const int64_t slot = p.slot_mapping[token];
  if (slot >= 0 && slot < p.num_slots) return slot;
  if (slot != -1 && report) flag_error(p.err, PKV_DEVERR_BAD_SLOT);
  return -1;
}

__device__ __forceinline__ int64_t tile_offset(int64_t slot, int32_t hkv, int32_t head) {
  const int64_t block = slot / kBlockSize;
  const int tile = static_cast<int>(slot % kBlockSize) / kQ4Tile;
  return (block * hkv + head) * kQ4RecordBytes + tile * kQ4TileBytes;
}

template <Elem E, bool kAligned>
__global__ void __launch_bounds__(kThreads, 5) store_q4_kernel(const Q4RowsParams p) {
  const int lane8 = threadIdx.x & 7, j = lane8 >> 1, u = lane8 & 1;
  const int head = static_cast<int>(blockIdx.x);
  const int64_t token = (static_cast<int64_t>(blockIdx.z) * p.blocks_per_z + blockIdx.y) * kRowsPerBlock +
                        (threadIdx.x >> 3);
  const int64_t slot = row_slot(p, token, lane8 == 0 && head == 0);
  uint4 kr[2], vr[2];
  kr[0] = kr[1] = vr[0] = vr[1] = make_uint4(0, 0, 0, 0);
  if (slot >= 0) {
    const uint16_t* ks = p.k + token * p.k_stride + head * kHeadDim + 32 * j + 8 * u;
    const uint16_t* vs = p.v + token * p.v_stride + head * kHeadDim + 32 * j + 8 * u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      kr[i] = kAligned ? ld_rows_v4(ks + 16 * i) : ld_rows_u16(ks + 16 * i);
      vr[i] = kAligned ? ld_rows_v4(vs + 16 * i) : ld_rows_u16(vs + 16 * i);
    }
  }
  uint32_t kp, vp, kc[2], vc[2];
  quantise16<E>(kr[0], kr[1], kp, kc[0], kc[1]);
  quantise16<E>(vr[0], vr[1], vp, vc[0], vc[1]);
  v_exchange2(vc[0], vc[1], j);
  if (slot < 0) return;
  const int tok = static_cast<int>(slot % kQ4Tile);
  const int64_t off = tile_offset(slot, p.hkv, head);
  uint8_t* kd = p.k_cache + off;
  uint8_t* vd = p.v_cache + off;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<uint32_t*>(kd + q4_k_word(tok, j, u + 2 * i)) = kc[i];
    *reinterpret_cast<uint32_t*>(vd + q4_v_word(tok, j, u + 2 * i)) = vc[i];
  }
  *reinterpret_cast<uint32_t*>((u == 0 ? kd : vd) + q4_param(tok, j)) = u == 0 ? kp : vp;
}

template <Elem E>
__global__ void __launch_bounds__(kThreads) load_q4_kernel(const Q4RowsParams p) {
  const int lane8 = threadIdx.x & 7, j = lane8 >> 1, u = lane8 & 1;
  const int head = static_cast<int>(blockIdx.x);
  const int64_t token = (static_cast<int64_t>(blockIdx.z) * p.blocks_per_z + blockIdx.y) * kRowsPerBlock +
                        (threadIdx.x >> 3);
  const int64_t slot = row_slot(p, token, lane8 == 0 && head == 0);
  uint32_t kc[2] = {0, 0}, vc[2] = {0, 0}, kp = 0, vp = 0;
  if (slot >= 0) {
    const int tok = static_cast<int>(slot % kQ4Tile);
    const int64_t off = tile_offset(slot, p.hkv, head);
    const uint8_t* ks = p.k_cache + off;
    const uint8_t* vs = p.v_cache + off;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      kc[i] = *reinterpret_cast<const uint32_t*>(ks + q4_k_word(tok, j, u + 2 * i));
      vc[i] = *reinterpret_cast<const uint32_t*>(vs + q4_v_word(tok, j, u + 2 * i));
    }
    kp = *reinterpret_cast<const uint32_t*>(ks + q4_param(tok, j));
    vp = *reinterpret_cast<const uint32_t*>(vs + q4_param(tok, j));
  }
  v_exchange2(vc[0], vc[1], j);
  if (slot < 0) return;
  const int64_t row = (token * p.hkv + head) * kHeadDim + 32 * j + 8 * u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<uint4*>(p.k_out + row + 16 * i) = dequantise8<E>(kc[i], kp);
    *reinterpret_cast<uint4*>(p.v_out + row + 16 * i) = dequantise8<E>(vc[i], vp);
  }
}

dim3 rows_grid(Q4RowsParams& p) {
  const int64_t nb = (static_cast<int64_t>(p.num_tokens) + kRowsPerBlock - 1) / kRowsPerBlock;
  p.blocks_per_z = static_cast<int32_t>(nb < 65535 ? nb : 65535);
  return dim3(static_cast<unsigned>(p.hkv), static_cast<unsigned>(p.blocks_per_z),
              static_cast<unsigned>((nb + p.blocks_per_z - 1) / p.blocks_per_z));
}

}  // namespace

cudaError_t launch_store_q4(const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* k_cache,
                            void* v_cache, const int32_t* slot_mapping, int32_t num_tokens, int32_t hkv,
                            int64_t num_slots, unsigned int* err, cudaStream_t stream, Elem elem) {
  Q4RowsParams p{};
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.slot_mapping = slot_mapping;
  p.num_slots = num_slots;
  p.num_tokens = num_tokens;
  p.hkv = hkv;
  p.err = err;
  const dim3 grid = rows_grid(p);
  const bool aligned = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) == 0 &&
                       k_stride % 8 == 0 && v_stride % 8 == 0;
  if (elem == Elem::kF16) {
    if (aligned)
      store_q4_kernel<Elem::kF16, true><<<grid, kThreads, 0, stream>>>(p);
    else
      store_q4_kernel<Elem::kF16, false><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (aligned)
      store_q4_kernel<Elem::kBF16, true><<<grid, kThreads, 0, stream>>>(p);
    else
      store_q4_kernel<Elem::kBF16, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_load_q4(const void* k_cache, const void* v_cache, const int32_t* slot_mapping, int32_t num_tokens,
                           int32_t hkv, int64_t num_slots, void* k, void* v, unsigned int* err, cudaStream_t stream,
                           Elem elem) {
  Q4RowsParams p{};
  p.k_out = static_cast<uint16_t*>(k);
  p.v_out = static_cast<uint16_t*>(v);
  p.k_cache = static_cast<uint8_t*>(const_cast<void*>(k_cache));
  p.v_cache = static_cast<uint8_t*>(const_cast<void*>(v_cache));
  p.slot_mapping = slot_mapping;
  p.num_slots = num_slots;
  p.num_tokens = num_tokens;
  p.hkv = hkv;
  p.err = err;
  const dim3 grid = rows_grid(p);
  if (elem == Elem::kF16)
    load_q4_kernel<Elem::kF16><<<grid, kThreads, 0, stream>>>(p);
  else
    load_q4_kernel<Elem::kBF16><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pkv
