// latent_cache.hip -- rows of the paged latent cache: append (norm, rotary
// part, paged write, and the queries' rotary part in the same launch) and keep
// (the accepted nodes' rows of a drafted tree, moved together).
#include "dev_attn.h"

namespace coli {
namespace {

using dev::u32x4;

// Append.  One 256-thread workgroup per token:
//   latent   y = c / sqrt(mean(c^2) + eps) * weight, over the 512 latent values
//   rotary   pairs (a, b) -> (a cos - b sin, a sin + b cos), pairs (2i, 2i + 1)
//            or (i, i + 32), of the row's 64 rotary values and of every head's
// The first wave owns the row: eight latent values per lane, the mean by a
// wave sum; all waves rotate 16-value parts (a quarter of a head) of the
// queries.  Everything is computed in fp32 and rounded once.  Bound by HBM: 8192
// tokens with 64 heads, 155 MB, in 24.5 us, 6.3 TB/s; 64 tokens 3.6 us, a launch.
constexpr int kAppendThreads = 256;

template <bool BF>
__device__ __forceinline__ void unpack8(u32x4 w, float (&v)[8]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        v[2 * d] = dev::lo16<BF>(w[d]);
        v[2 * d + 1] = dev::hi16<BF>(w[d]);
    }
}
template <bool BF>
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
    return u32x4{dev::pack2<BF>(v[0], v[1]), dev::pack2<BF>(v[2], v[3]), dev::pack2<BF>(v[4], v[5]), dev::pack2<BF>(v[6], v[7])};
}

// Part `part` (of four) of one 64-value rotary vector: pairs 8 part .. + 7,
// which are values 16 part .. + 15 (interleaved) or 8 part .. + 7 and the same
// 32 further (halves).
template <bool BF>
__device__ __forceinline__ void rotate_part(const uint8_t *src, uint8_t *dst, int part, const float *cs, const float *sn,
                                            bool interleaved) {
    const int at0 = interleaved ? 32 * part : 16 * part, at1 = interleaved ? at0 + 16 : at0 + 64;   // bytes
    float x[8], y[8], c[8], s[8];
    unpack8<BF>(*reinterpret_cast<const u32x4 *>(src + at0), x);
    unpack8<BF>(*reinterpret_cast<const u32x4 *>(src + at1), y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = cs[8 * part + i];
        s[i] = sn[8 * part + i];
    }
    float u[8], v[8];
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
            u[2 * i + 1] = x[2 * i] * s[i] + x[2 * i + 1] * c[i];
            v[2 * i] = y[2 * i] * c[4 + i] - y[2 * i + 1] * s[4 + i];
            v[2 * i + 1] = y[2 * i] * s[4 + i] + y[2 * i + 1] * c[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u[i] = x[i] * c[i] - y[i] * s[i];
            v[i] = x[i] * s[i] + y[i] * c[i];
        }
    }
    *reinterpret_cast<u32x4 *>(dst + at0) = pack8<BF>(u);
    *reinterpret_cast<u32x4 *>(dst + at1) = pack8<BF>(v);
}

template <bool BF>
__global__ __launch_bounds__(kAppendThreads) void append_kernel(AppendArgs a) {
    const int t = blockIdx.x, tid = threadIdx.x;
    int pos = a.pos[t];
    const bool bad_pos = pos < 0 || pos >= a.n_pos;
    if (bad_pos) pos = 0;
    const float *cs = a.cos_t + static_cast<int64_t>(pos) * (kRope / 2), *sn = a.sin_t + static_cast<int64_t>(pos) * (kRope / 2);
    if (tid < 64) {
        const int64_t slot = a.slots[t];
        const int64_t page = slot >> a.page_shift;
        const bool bad_slot = slot >= 0 && page >= a.n_pages;
        dev::flag_if(tid == 0 && (bad_slot || bad_pos), a.err, kErrPage);
        if (slot >= 0 && !bad_slot && !bad_pos) {
            const uint8_t *c = a.c + static_cast<int64_t>(t) * a.c_stride * 2;
            uint8_t *row = a.cache + (page * a.page_stride + (slot & ((1ll << a.page_shift) - 1)) * kCacheRow) * 2;
            float v[8], w[8];
            unpack8<BF>(*reinterpret_cast<const u32x4 *>(c + 16 * tid), v);
            unpack8<BF>(*reinterpret_cast<const u32x4 *>(a.weight + 16 * tid), w);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(v[i], v[i], sum);
#pragma unroll
            for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o, 64);
            const float by = 1.0f / __builtin_sqrtf(sum * (1.0f / kLatent) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * by * w[i];
            *reinterpret_cast<u32x4 *>(row + 16 * tid) = pack8<BF>(v);
            if (tid < 4) rotate_part<BF>(c + 2 * kLatent, row + 2 * kLatent, tid, cs, sn, a.interleaved);
        }
    }
    if (a.q_pe) {
        const uint8_t *q = a.q_pe + static_cast<int64_t>(t) * a.q_tok * 2;
        uint8_t *o = a.q_out + static_cast<int64_t>(t) * a.n_heads * kRope * 2;
        for (int u = tid; u < 4 * a.n_heads; u += kAppendThreads)
            rotate_part<BF>(q + (u >> 2) * a.q_head * 2, o + (u >> 2) * kRope * 2, u & 3, cs, sn, a.interleaved);
    }
}

// Keep.  A tree's nodes occupy the last rows of their sequence in node order;
// path[i] is the node that row i of them becomes.  path ascends, so path[i] >=
// i and moving the rows in order never overwrites one still to be read.  A
// thread owns one 16-byte unit of the rows of one (layer, sequence) and
// moves it for eight path entries at a time: their loads are in flight
// together, the stores follow.  Bound by the chain of dependent loads (path, page,
// row): 16 sequences of one layer 5.2 us, 128 of 12 layers, 18 MB, 8.4 us.
constexpr int kKeepThreads = 256;
constexpr int kRowUnits = kCacheRow * 2 / 16;
constexpr int kKeepBatch = 8;

__global__ __launch_bounds__(kKeepThreads) void keep_kernel(KeepArgs a, int64_t units) {
    const int64_t g = static_cast<int64_t>(blockIdx.x) * kKeepThreads + threadIdx.x;
    if (g >= units) return;
    const int unit = static_cast<int>(g % kRowUnits);
    const int64_t rest = g / kRowUnits;
    const int b = static_cast<int>(rest % a.n_seq);
    const int64_t layer = rest / a.n_seq;
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1], len = a.kv_len[b];
    const int n = q1 - q0, base = len - n;
    const bool report = unit == 0 && layer == 0;
    if (q0 < 0 || n < 0 || q1 > a.n_tok || base < 0) {
        dev::flag_if(report, a.err, kErrSeq);
        return;
    }
    const int32_t *table = a.cache.table + b * a.cache.table_stride;
    const int32_t *path = a.path + b * a.path_stride;
    uint8_t *cache = a.cache.base + (layer * a.layer_stride) * 2 + 16 * unit;
    auto row_of = [&](int node) -> uint8_t * {
        const int pos = base + node, at = pos >> a.cache.page_shift;
        const int page = at < a.cache.table_cols ? table[at] : -1;
        if (page < 0 || page >= a.cache.n_pages) return nullptr;
        return cache + (page * a.cache.page_stride + static_cast<int64_t>(pos & ((1 << a.cache.page_shift) - 1)) * kCacheRow) * 2;
    };
    bool bad = false, bad_page = false, more = true;
    const int cols = min(a.path_cols, n);
    for (int i0 = 0; i0 < cols && more; i0 += kKeepBatch) {
        u32x4 v[kKeepBatch];
        uint8_t *to[kKeepBatch];
#pragma unroll
        for (int j = 0; j < kKeepBatch; ++j) {
            to[j] = nullptr;
            const int i = i0 + j;
            const int node = i < cols ? path[i] : -1;
            more = more && node >= 0;
            if (more && (node >= n || node < i)) {
                bad = true;
                more = false;
            }
            if (!more || node == i) continue;
            const uint8_t *from = row_of(node);
            uint8_t *dst = row_of(i);
            if (!from || !dst) {
                bad_page = true;
                continue;
            }
            to[j] = dst;
            v[j] = *reinterpret_cast<const u32x4 *>(from);
        }
#pragma unroll
        for (int j = 0; j < kKeepBatch; ++j)
            if (to[j]) *reinterpret_cast<u32x4 *>(to[j]) = v[j];
    }
    dev::flag_if(report && bad, a.err, kErrDraft);
    dev::flag_if(report && bad_page, a.err, kErrPage);
}

}  // namespace

hipError_t launch_append(const AppendArgs &a, bool bf16, hipStream_t s) {
    launch(bf16 ? append_kernel<true> : append_kernel<false>, static_cast<unsigned>(a.n_tok), kAppendThreads, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_keep(const KeepArgs &a, hipStream_t s) {
    const int64_t units = static_cast<int64_t>(a.n_layers) * a.n_seq * kRowUnits;
    const int64_t blocks = (units + kKeepThreads - 1) / kKeepThreads;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    launch(keep_kernel, static_cast<unsigned>(blocks), kKeepThreads, 0, s, a, units);
    return hipGetLastError();
}

}  // namespace coli
