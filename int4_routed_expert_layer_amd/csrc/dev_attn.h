// dev_attn.h -- device helpers of the latent-attention kernels: 16-bit
// fragments on v_mfma_f32_32x32x16, the swizzled LDS tile, transposed reads.
#pragma once

#include "dev_common.h"
#include "serve.h"

namespace coli {
namespace dev {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// D = A B + C on 32 x 32 x 16: lane L holds A[m = L % 32][k = 8 (L / 32) + j],
// B[k = 8 (L / 32) + j][n = L % 32], j = 0..7, and
// D[m = 8 (i / 4) + 4 (L / 32) + i % 4][n = L % 32], i = 0..15.
template <bool BF>
__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two fp32 values rounded (to nearest even) to one dword of 16-bit values.
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF) {
        const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
        return __builtin_bit_cast(uint32_t, v);
    } else {
        const f16x2 v = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
        return __builtin_bit_cast(uint32_t, v);
    }
}
template <bool BF>
__device__ __forceinline__ float lo16(uint32_t w) {
    if constexpr (BF) return __uint_as_float(w << 16);
    return static_cast<float>(__builtin_bit_cast(f16x2, w)[0]);
}
template <bool BF>
__device__ __forceinline__ float hi16(uint32_t w) {
    if constexpr (BF) return __uint_as_float(w & 0xFFFF0000u);
    return static_cast<float>(__builtin_bit_cast(f16x2, w)[1]);
}

// All-ones in each 16-bit half of w whose value is inf or NaN: adding one to
// an all-ones exponent carries into the (cleared) sign bit.
template <bool BF>
__device__ __forceinline__ uint32_t nonfinite_halves(uint32_t w) {
    constexpr uint32_t kExp = BF ? 0x7F807F80u : 0x7C007C00u, kOne = BF ? 0x00800080u : 0x04000400u;
    const uint32_t c = (((w & kExp) + kOne) & 0x80008000u) >> 15;
    return c * 0xFFFFu;
}

// LDS tiles hold 64 rows of 128 bytes (64 values), rows of one 64-column
// block after each other.  The 16-byte unit q of row r lies at unit
// q ^ tile_swz(r): with 64 banks of four bytes a row covers half of them, so
// 16 consecutive rows read at one unit (fragment reads) cover every bank once,
// and so do four consecutive rows read at four adjacent units (transposed
// reads): the bit of r that separates row pairs flips the unit's highest bit.
__device__ __forceinline__ int tile_swz(int r) {
    const int p = (r >> 1) & 7;
    return ((p & 1) << 2) | (p & 2) | (p >> 2);
}
__device__ __forceinline__ int tile_unit(int r, int q) { return r * 128 + ((q ^ tile_swz(r)) << 4); }

// Transposed read: each 16-lane group reads a 4 x 16 block (lane i gives the
// address of row i / 4, columns 4 (i % 4) .. + 3) and lane i gets column i of
// its four rows.
__device__ __forceinline__ u32x2 read_tr(const uint8_t *p) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4 *)(const_cast<uint8_t *>(p)));
    return __builtin_bit_cast(u32x2, v);
}

// Workgroup barrier that waits for this wave's LDS accesses but not for its
// global loads in flight (__syncthreads would).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// The same after every global load and copy into LDS of this wave has landed.
__device__ __forceinline__ void copy_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Stores 32 columns x 32 rows of an accumulator as 16-bit values: lane L holds
// row L % 32 and columns 8 g + 4 (L / 32) + 0..3 in registers 4 g .. 4 g + 3;
// the lanes of a row trade halves so that each stores 16 bytes.  `row` is the
// lane's row at the tile's first column, NULL for a row that is not stored.
template <bool BF>
__device__ __forceinline__ void store_tile16(const f32x16 &acc, float by, uint8_t *row) {
    const int lh = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
        uint32_t w[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int d = 0; d < 2; ++d)
                w[k][d] = pack2<BF>(acc[4 * (g + k) + 2 * d] * by, acc[4 * (g + k) + 2 * d + 1] * by);
        const auto a = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
        if (row) *reinterpret_cast<u32x4 *>(row + 16 * (g + lh)) = u32x4{a[0], b[0], a[1], b[1]};
    }
}

}  // namespace dev
}  // namespace coli
