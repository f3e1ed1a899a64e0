// What the tensor-core window-attention kernels share: swizzled row tiles, the
// two kinds of product they issue, and the tensor maps of strided head rows.
#pragma once

#include "attn_math.cuh"
#include "sm100.cuh"

namespace ccgqa {
namespace {

// Rows of d bf16 in shared memory: panels of 64 (d = 32: 32) columns, each row of
// a panel one swizzle row.
template <int D>
struct RowTiles {
  static constexpr int kPanelCols = D == 32 ? 32 : 64;
  static constexpr int kPanels = D / kPanelCols;
  static constexpr uint32_t kRowBytes = kPanelCols * 2;
  static constexpr uint32_t kSwz = D == 32 ? sm100::kSwizzle64B : sm100::kSwizzle128B;
  static constexpr uint32_t kSbo = 8 * kRowBytes;             // 8-row group stride
};

// acc = A B^T over d: A 128 rows at a_base, B rows at b_base (as many as idesc
// says), panels a_panel and b_panel bytes apart.
template <int D>
__device__ __forceinline__ void mma_rows_by_rows(uint32_t acc, uint32_t a_base, uint32_t a_panel, uint32_t b_base,
                                                 uint32_t b_panel, uint32_t idesc) {
  using R = RowTiles<D>;
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const int p = k * 16 / R::kPanelCols;
    const uint32_t in = k * 16 % R::kPanelCols * 2;
    sm100::mma_ss(acc, sm100::make_smem_desc(a_base + p * a_panel + in, 16, R::kSbo, R::kSwz),
                  sm100::make_smem_desc(b_base + p * b_panel + in, 16, R::kSbo, R::kSwz), idesc, k > 0 ? 1u : 0u);
  }
}

// acc (+)= A B: A 128 x N bf16 in TMEM, B N rows at b_base read MN-major.
template <int D, int N>
__device__ __forceinline__ void mma_tmem_by_rows(uint32_t acc, uint32_t a_tmem, uint32_t b_base, uint32_t b_panel,
                                                 uint32_t idesc, bool first) {
  using R = RowTiles<D>;
#pragma unroll
  for (int k = 0; k < N / 16; ++k)
    sm100::mma_ts(acc, a_tmem + k * 8, sm100::make_smem_desc(b_base + k * 16 * R::kRowBytes, b_panel, R::kSbo, R::kSwz),
                  idesc, !first || k > 0 ? 1u : 0u);
}

// Bits [0, n) of a 64-bit set, n clamped to [0, 64].
__device__ __forceinline__ uint64_t below(int n) {
  return n >= 64 ? ~uint64_t(0) : (n <= 0 ? 0 : (uint64_t(1) << n) - 1);
}
__device__ __forceinline__ uint32_t below32(int n) {
  return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1);
}

// 32 fp32 values times f of each lane's row, as bf16, to 64 contiguous bytes at
// the lane's dst (null: no store).  The warp turns them in 2 KB of shared memory
// (16-byte units exchanged against bank conflicts) so that four lanes write a
// row's 64 bytes: stored straight from their rows, 32 lines a store, a 128 x 128
// tile took 4000 cycles.
__device__ __forceinline__ void warp_store32(bf16* dst, const uint32_t (&v)[32], float f, uint8_t* stage, int lane) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16x2(__uint_as_float(v[u * 8 + 2 * e]) * f, __uint_as_float(v[u * 8 + 2 * e + 1]) * f);
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((u ^ (lane >> 1)) & 3) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i * 8 + (lane >> 2), u = lane & 3;
    const uint4 w = *reinterpret_cast<const uint4*>(stage + row * 64 + ((u ^ (row >> 1)) & 3) * 16);
    bf16* p = reinterpret_cast<bf16*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
    if (p != nullptr) *reinterpret_cast<uint4*>(p + u * 8) = w;
  }
  __syncwarp();
}

// 32 bytes of each lane's row, likewise, two lanes a row.
__device__ __forceinline__ void warp_store_bytes32(int8_t* dst, const uint32_t (&w)[8], uint8_t* stage, int lane) {
#pragma unroll
  for (int u = 0; u < 2; ++u)
    *reinterpret_cast<uint4*>(stage + lane * 32 + ((u ^ (lane >> 2)) & 1) * 16) =
        make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = i * 16 + (lane >> 1), u = lane & 1;
    const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 32 + ((u ^ (row >> 2)) & 1) * 16);
    int8_t* p = reinterpret_cast<int8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
    if (p != nullptr) *reinterpret_cast<uint4*>(p + u * 16) = x;
  }
  __syncwarp();
}

// Rows of `tiles` tiles of `rows` rows that the packed TMA box does not fill
// (the group does not divide the tile): zeros, so that their products are
// finite.  Called by all threads before the first product.
template <int D>
__device__ __forceinline__ void zero_unused_rows(uint8_t* base, int tiles, int rows, int rows_used) {
  using R = RowTiles<D>;
  if (rows_used >= rows) return;
  const int n16 = (rows - rows_used) * static_cast<int>(R::kRowBytes) / 16;
  for (int i = threadIdx.x; i < tiles * R::kPanels * n16; i += blockDim.x) {
    const int tp = i / n16, w = i % n16;
    *reinterpret_cast<uint4*>(base + (tp * rows + rows_used) * R::kRowBytes + w * 16) = make_uint4(0, 0, 0, 0);
  }
  sm100::fence_proxy_async_smem();
}

// After an abandoned wait: TMEM is not released while a product may write it.
__device__ __forceinline__ void drain_mmas(uint64_t* drain) {
  sm100::mma_commit(drain);
  const long long t0 = clock64();
  while (!sm100::mbar_try_wait(drain, 0) && clock64() - t0 < kWaitLimitCycles) {
  }
}

inline uint64_t map_stride(int64_t elements, int64_t n) {
  return n > 1 ? static_cast<uint64_t>(elements) * 2 : 16;   // a dimension of one needs any valid stride
}
inline CUtensorMapSwizzle map_swizzle(int d) {
  return d == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
}
// Query rows [B, S, Hq, d] as (d, G, Hkv, S, B): a box (panel, G, 1, pos, 1)
// lands as pos G packed rows (position, head in group).
inline bool packed_rows_map(CUtensorMap* m, const Rows& r, const WindowArgs& a, int pos) {
  const uint64_t dims[5] = {static_cast<uint64_t>(a.d), static_cast<uint64_t>(a.G), static_cast<uint64_t>(a.Hkv),
                            static_cast<uint64_t>(a.S), static_cast<uint64_t>(a.B)};
  const uint64_t st[4] = {map_stride(r.head, a.G), map_stride(r.head * a.G, a.Hkv), map_stride(r.token, a.S),
                          map_stride(r.batch, a.B)};
  const uint32_t box[5] = {a.d == 32 ? 32u : 64u, static_cast<uint32_t>(a.G), 1, static_cast<uint32_t>(pos), 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, r.ptr, dims, st, box, map_swizzle(a.d));
}
// Key rows [B, S, Hkv, d] as (d, S, Hkv, B) in boxes of `rows` tokens.
inline bool key_rows_map(CUtensorMap* m, const Rows& r, const WindowArgs& a, int rows) {
  const uint64_t dims[4] = {static_cast<uint64_t>(a.d), static_cast<uint64_t>(a.S), static_cast<uint64_t>(a.Hkv),
                            static_cast<uint64_t>(a.B)};
  const uint64_t st[3] = {map_stride(r.token, a.S), map_stride(r.head, a.Hkv), map_stride(r.batch, a.B)};
  const uint32_t box[4] = {a.d == 32 ? 32u : 64u, static_cast<uint32_t>(rows), 1, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, r.ptr, dims, st, box, map_swizzle(a.d));
}

}  // namespace
}  // namespace ccgqa
