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
typedef float f32x2 __attribute__((ext_vector_type(2)));
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

// D = A B + C on 16 x 16 x 32: lane L holds A[m = L % 16][k = 8 (L / 16) + j],
// B[k = 8 (L / 16) + j][n = L % 16] and D[m = 4 (L / 16) + i][n = L % 16], i = 0..3.
template <bool BF>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
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

// LDS tiles hold rows of 128 bytes (64 values), the rows of one 64-column block
// after each other.  The 16-byte unit q of row r lies at unit q ^ ((r >> 1) & 7).
// Measured with eight waves reading, this is free of conflicts (4.6 clocks per
// 1 KB read of a wave) for the fragment reads of both MFMA shapes and for
// transposed reads; r & 7 costs 7.2 in 32-row fragments, and an order that
// flips the unit's highest bit between row pairs 7.3 in 16-row ones.
__device__ __forceinline__ int tile_swz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int tile_unit(int r, int q) { return r * 128 + ((q ^ tile_swz(r)) << 4); }

// Sum of the lanes up to this one, in the registers (shuffles by way of LDS take
// six latencies of it).
__device__ __forceinline__ int running_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1 .. 8 within 16 lanes
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
    return v;
}

// Transposed read: each 16-lane group reads a 4 x 16 block (lane i gives the
// address of row i / 4, columns 4 (i % 4) .. + 3) and lane i gets column i of
// its four rows.
__device__ __forceinline__ u32x2 read_tr(const uint8_t *p) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4 *)(const_cast<uint8_t *>(p)));
    return __builtin_bit_cast(u32x2, v);
}

// A value's maximum or sum over the two lanes L and L + 32 that share a row.
__device__ __forceinline__ float max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The same over lanes 0-15 and 16-31, 32-47 and 48-63.
__device__ __forceinline__ float max_quarters(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_quarters(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// copy16_to_lds (see dev_common.h) that the compiler may move among accesses
// it does not depend on, between the barriers around it: the caller fills a
// buffer that nothing reads before the next barrier.
__device__ __forceinline__ void copy16_to_lds_free(const void *src, uint32_t lds_addr) {
    asm volatile("global_load_lds_dwordx4 %0, off" ::"v"(src), "{m0}"(lds_addr));
}

// The same for data read once (non-temporal).
__device__ __forceinline__ void copy16_to_lds_once(const void *src, uint32_t lds_addr) {
    asm volatile("global_load_lds_dwordx4 %0, off nt" ::"v"(src), "{m0}"(lds_addr));
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

// Scheduling of the block they end: AHEAD LDS reads first, then READS reads
// after every MFMAS products, so that a read is issued while the products
// before its own are in the matrix pipe.
template <int AHEAD>
__device__ __forceinline__ void pipeline_begin() {
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
}
template <int LEFT, int MFMAS, int READS>
__device__ __forceinline__ void pipeline_run() {
    if constexpr (LEFT > 0) {
        __builtin_amdgcn_sched_group_barrier(0x008, MFMAS, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, LEFT < READS ? LEFT : READS, 0);
        pipeline_run<LEFT - READS, MFMAS, READS>();
    }
}
template <int READS_ALL, int MFMAS, int READS, int AHEAD>
__device__ __forceinline__ void pipeline() {
    pipeline_begin<AHEAD>();
    pipeline_run<READS_ALL - AHEAD, MFMAS, READS>();
}

// Sixteen bytes of a 32 x 32 accumulator as 16-bit values: lane L holds row L %
// 32 and columns 8 g + 4 (L / 32) + 0..3 in registers 4 g .. 4 g + 3; the lanes
// of a row trade halves, and L gets columns 8 (G + L / 32) .. + 7.
template <bool BF, int G>
__device__ __forceinline__ u32x4 pack_tile16(const f32x16 &acc, float by) {
    uint32_t w[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int d = 0; d < 2; ++d)
            w[k][d] = pack2<BF>(acc[4 * (G + k) + 2 * d] * by, acc[4 * (G + k) + 2 * d + 1] * by);
    const auto a = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
    return u32x4{a[0], b[0], a[1], b[1]};
}
// Stores 32 columns x 32 rows.  `row` is the lane's row at the tile's first
// column, NULL for a row that is not stored.
template <bool BF>
__device__ __forceinline__ void store_tile16(const f32x16 &acc, float by, uint8_t *row) {
    const int lh = (threadIdx.x & 63) >> 5;
    const u32x4 x = pack_tile16<BF, 0>(acc, by), y = pack_tile16<BF, 2>(acc, by);
    if (!row) return;
    *reinterpret_cast<u32x4 *>(row + 16 * lh) = x;
    *reinterpret_cast<u32x4 *>(row + 16 * (2 + lh)) = y;
}
// Stores 64 columns x 32 rows by way of 4 KB of LDS that the wave has to itself,
// 128 bytes of a row together (as 32 bytes of 32 rows each store occupies the
// CU's address unit longer: 32 prompts of 128 rows, 64 heads, 256 columns 167 us,
// so 137; 128 columns 76 and 71).  `by` is of the lane's row L % 32, `at` row 0,
// `rows` the rows stored, `stride` their distance in bytes.
template <bool BF>
__device__ __forceinline__ void store_rows16(const f32x16 &acc0, const f32x16 &acc1, float by, uint8_t *lds, uint8_t *at, int64_t stride, int rows) {
    int lane = threadIdx.x & 63;
    // What the area held before has been read.  Nor does the compiler see that
    // the lane's addresses here are like those of a caller's loop: it would hold
    // their parts in registers across it (500 spilled ones in the narrow head).
    asm volatile("" : "+v"(lane)::"memory");
    const int l31 = lane & 31, lh = lane >> 5;
    *reinterpret_cast<u32x4 *>(lds + tile_unit(l31, lh)) = pack_tile16<BF, 0>(acc0, by);
    *reinterpret_cast<u32x4 *>(lds + tile_unit(l31, 2 + lh)) = pack_tile16<BF, 2>(acc0, by);
    *reinterpret_cast<u32x4 *>(lds + tile_unit(l31, 4 + lh)) = pack_tile16<BF, 0>(acc1, by);
    *reinterpret_cast<u32x4 *>(lds + tile_unit(l31, 6 + lh)) = pack_tile16<BF, 2>(acc1, by);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    u32x4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const u32x4 *>(lds + tile_unit(8 * j + (lane >> 3), lane & 7));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 8 * j + (lane >> 3);
        if (r < rows) *reinterpret_cast<u32x4 *>(at + r * stride + 16 * (lane & 7)) = v[j];
    }
}

}  // namespace dev
}  // namespace coli
