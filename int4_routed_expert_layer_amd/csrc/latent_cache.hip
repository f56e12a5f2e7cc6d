// latent_cache.hip -- rows of the paged latent cache, of 16 or 8 bits: append (norm,
// rotary part, paged write, and the queries' rotary part in the same launch), read
// (contexts as 16-bit rows), keep (the accepted nodes' rows of a drafted tree,
// moved together) and reorder (the rows and tables of the beams that go on).
#include <type_traits>

#include "dev_attn.h"

namespace coli {
namespace {

using dev::u32x2;
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

// Eight of a row's latent values, four lanes to a group of 32, into a row of an 8-bit
// cache: v = q 2^k with q in e4m3, rounded once (to nearest even).  k is the least
// exponent that brings the group's values to 448, the largest e4m3, or below; as e4m3
// has the same relative precision over 15 powers of two, a scale that is a power of
// two loses none of it, and every q 2^k is a value of the 16-bit type, so that reading
// is exact.  That bounds k: from below where the least step of q, 2^-9, would leave the
// type (f16) or its normal numbers (bf16), and from above where 448 would: there
// values end at 240.  8192 tokens with 64 heads, 151 MB: 28.6 us, 5.3 TB/s; 64 tokens 3.8, a
// launch.  A value that is not finite in the 16-bit type is stored as NaN and
// has no part in the scale.
template <bool BF>
__device__ __forceinline__ void store8(const float (&v)[8], uint8_t *row, int lane) {
    constexpr int kLeast = BF ? -110 : -15, kMost = BF ? 120 : 8;
    const u32x4 half = pack8<BF>(v);
    uint32_t off[4];
    float most = 0.0f;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        off[d] = dev::nonfinite_halves<BF>(half[d]);
        most = fmaxf(most, fmaxf(off[d] & 0xFFFFu ? 0.0f : fabsf(v[2 * d]), off[d] >> 16 ? 0.0f : fabsf(v[2 * d + 1])));
    }
    most = fmaxf(most, __shfl_xor(most, 1, 64));
    most = fmaxf(most, __shfl_xor(most, 2, 64));
    const uint32_t bits = __float_as_uint(most);
    int k = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // 448 = 1.75 2^8
    k = min(max(k, kLeast), kMost);
    const float by = __uint_as_float(static_cast<uint32_t>(127 - k) << 23), end = k == kMost ? 240.0f : 448.0f;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool gone = (i & 1 ? off[i >> 1] >> 16 : off[i >> 1] & 0xFFFFu) != 0;
        q[i] = gone ? __builtin_nanf("") : fminf(fmaxf(v[i] * by, -end), end);
    }
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
        w[h] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], lo, true));
    }
    *reinterpret_cast<u32x2 *>(row + 8 * lane) = w;
    if ((lane & 3) == 0) row[kRow8Scales + (lane >> 2)] = static_cast<uint8_t>(k + 127);
}

template <bool BF, bool Q8>
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
            uint8_t *row = a.cache + page * a.page_bytes + (slot & ((1ll << a.page_shift) - 1)) * (Q8 ? kRow8Bytes : kRowBytes);
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
            if constexpr (Q8) store8<BF>(v, row, tid);
            else *reinterpret_cast<u32x4 *>(row + 16 * tid) = pack8<BF>(v);
            if (tid < 4) rotate_part<BF>(c + 2 * kLatent, row + (Q8 ? kRow8Rope : 2 * kLatent), tid, cs, sn, a.interleaved);
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
constexpr int kKeepBatch = 8;
template <bool Q8>
constexpr int kRowUnits = (Q8 ? kRow8Bytes : kRowBytes) / 16;

template <bool Q8>
__global__ __launch_bounds__(kKeepThreads) void keep_kernel(KeepArgs a, int64_t units) {
    const int64_t g = static_cast<int64_t>(blockIdx.x) * kKeepThreads + threadIdx.x;
    if (g >= units) return;
    const int unit = static_cast<int>(g % kRowUnits<Q8>);
    const int64_t rest = g / kRowUnits<Q8>;
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
    uint8_t *cache = a.cache.base + layer * a.layer_bytes + 16 * unit;
    auto row_of = [&](int node) -> uint8_t * {
        const int pos = base + node, at = pos >> a.cache.page_shift;
        const int page = at < a.cache.table_cols ? table[at] : -1;
        if (page < 0 || page >= a.cache.n_pages) return nullptr;
        return cache + page * a.cache.page_bytes + static_cast<int64_t>(pos & ((1 << a.cache.page_shift) - 1)) * (Q8 ? kRow8Bytes : kRowBytes);
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

// Read.  Output row t is position first[b] + t - k_start[b] of the sequence b that it
// falls in.  A workgroup takes 8 rows: a wave finds their sequences (64 bounds at a time)
// and addresses, then each thread moves three 16-byte units of output.  Rows of 8 bits come
// by way of LDS, as they lie, and are converted from there: eight values and their scale
// loaded by each thread as it needs them, 16 rows a workgroup, took 97 us for what now
// takes 79.  Rows before the first sequence and behind the last are left alone.
// Sixteen contexts of 8787 to 32767 rows, 8 bits, 448 MB: 79 us, 5.7 TB/s; 16 of 16384, 16
// bits, 604 MB: 102 us, 5.9; eight up to 1023 rows 3.8 us, a chain of dependent loads
// (bound, page, row).  16 rows by 384 threads take the same; by 192 85 and 121, by 576 107 and
// 100; 8 rows by 288 98 and 104, 4 by 96 85 and 110.
constexpr int kReadRows = 8, kReadThreads = 192;
constexpr int kOutUnits = kRowBytes / 16, kReadEach = kReadRows * kOutUnits / kReadThreads;
static_assert(kReadEach * kReadThreads == kReadRows * kOutUnits, "whole rounds of units");

// With STREAM the stores bypass the caches: 16 contexts of 16384 rows, 16 bits, 113 us, so
// 102 (8 bits the same).  Of fewer bytes what comes next finds them there.
constexpr int64_t kStreamBytes = 64 << 20;

template <bool BF, bool Q8, bool STREAM>
__global__ __launch_bounds__(kReadThreads) void read_kernel(ReadArgs a) {
    __shared__ const uint8_t *s_row[kReadRows];
    const int tid = threadIdx.x;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kReadRows;
    if (tid < 64) {
        // The last sequence that begins at or before row0: 64 candidates a round.
        int lo = 0, n = a.n_seq;                          // it is among lo .. lo + n - 1
        while (n > 1) {
            const int step = (n + 63) / 64, at = lo + min(tid * step, n - 1);
            const uint64_t m = __ballot(a.k_start[at] <= row0);
            const int k = m ? 63 - __clzll(m) : 0;
            n = min(step, n - min(k * step, n - 1));
            lo = __builtin_amdgcn_readlane(at, k);
        }
        const int64_t t = row0 + (tid & (kReadRows - 1));
        bool bad = false, bad_page = false;
        const uint8_t *from = nullptr;
        if (tid < kReadRows && t < a.n_rows) {
            int b = lo, end = a.n_seq;                    // rows of one workgroup mostly share it
            if (b + 1 < end && a.k_start[b + 1] <= t)
                while (b + 1 < end) {
                    const int mid = b + (end - b) / 2;
                    if (a.k_start[mid] <= t) b = mid;
                    else end = mid;
                }
            const int k0 = a.k_start[b], k1 = a.k_start[b + 1];
            if (t >= k0 && t < k1) {
                const int64_t pos = (a.first ? a.first[b] : 0) + (t - k0);
                const int64_t at = pos >> a.cache.page_shift;
                bad = k0 < 0 || k1 > a.n_rows;
                const int page = pos >= 0 && at < a.cache.table_cols ? a.cache.table[b * a.cache.table_stride + at] : -1;
                bad_page = page < 0 || page >= a.cache.n_pages;
                if (!bad_page && !bad)
                    from = a.cache.base + page * a.cache.page_bytes + (pos & ((1ll << a.cache.page_shift) - 1)) * (Q8 ? kRow8Bytes : kRowBytes);
            } else {
                bad = k1 < k0 || (b > 0 && t < k0);       // bounds that do not ascend
            }
        }
        if (tid < kReadRows) s_row[tid] = from;
        dev::flag_if(bad, a.err, kErrSeq);
        dev::flag_if(bad_page, a.err, kErrPage);
    } else {
        // Meanwhile the other waves look for bounds that do not ascend: the search passes by
        // those of sequences that no row of its workgroup falls in.
        constexpr int kOthers = kReadThreads - 64;
        bool bad = false;
        for (int64_t b = static_cast<int64_t>(blockIdx.x) * kOthers + tid - 64; b < a.n_seq; b += static_cast<int64_t>(gridDim.x) * kOthers) {
            const int k0 = a.k_start[b], k1 = a.k_start[b + 1];
            bad = bad || k0 < 0 || k1 < k0 || k1 > a.n_rows;
        }
        dev::flag_if(bad, a.err, kErrSeq);
    }
    __syncthreads();
    auto load = [](auto *p) {
        typedef std::remove_const_t<std::remove_pointer_t<decltype(p)>> T;
        return *(const __attribute__((address_space(1))) T *)(p);
    };
    u32x4 v[kReadEach];
    uint32_t by[kReadEach];
    __shared__ __align__(16) uint8_t s_raw[Q8 ? kReadRows * kRow8Bytes : 16];
    if constexpr (Q8) {
        // The rows' bytes as they lie, by way of LDS.
        constexpr int kUnits = kRow8Bytes / 16, kEach = (kReadRows * kUnits + kReadThreads - 1) / kReadThreads;
        u32x4 raw[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int g = tid + i * kReadThreads, r = min(g / kUnits, kReadRows - 1), u = g - r * kUnits;
            const uint8_t *from = g < kReadRows * kUnits ? s_row[r] : nullptr;
            if (from) raw[i] = load(reinterpret_cast<const u32x4 *>(from + 16 * u));
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int g = tid + i * kReadThreads;
            if (g < kReadRows * kUnits) *reinterpret_cast<u32x4 *>(s_raw + 16 * g) = raw[i];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kReadEach; ++i) {
        const int g = tid + i * kReadThreads, r = g / kOutUnits, u = g - r * kOutUnits;
        const uint8_t *from = s_row[r];
        if (!from) continue;
        const uint8_t *raw = s_raw + r * kRow8Bytes;
        if constexpr (!Q8) {
            v[i] = load(reinterpret_cast<const u32x4 *>(from + 16 * u));
        } else if (u < kLatent / 8) {
            const u32x2 q = *reinterpret_cast<const u32x2 *>(raw + 8 * u);
            v[i] = u32x4{q[0], q[1], 0, 0};
            by[i] = raw[kRow8Scales + u / 4];
        } else {
            v[i] = *reinterpret_cast<const u32x4 *>(raw + kRow8Rope + 16 * (u - kLatent / 8));
        }
    }
#pragma unroll
    for (int i = 0; i < kReadEach; ++i) {
        const int g = tid + i * kReadThreads, r = g / kOutUnits, u = g - r * kOutUnits;
        if (!s_row[r]) continue;
        u32x4 w = v[i];
        if (Q8 && u < kLatent / 8) {
            const float f = __uint_as_float(by[i] << 23);
            w = u32x4{dev::of_fp8<BF, false>(v[i][0], f), dev::of_fp8<BF, true>(v[i][0], f), dev::of_fp8<BF, false>(v[i][1], f), dev::of_fp8<BF, true>(v[i][1], f)};
        }
        u32x4 *to = reinterpret_cast<u32x4 *>(a.out + (row0 + r) * a.out_stride * 2 + 16 * u);
        if constexpr (STREAM) __builtin_nontemporal_store(w, to);
        else *to = w;
    }
}

// Reorder.  Place j of a group goes on as beam p = parents[j].  Whole pages are never
// written again, so places share them; the page that the next token is written to has
// to be a place's own.  The first place that continues a beam keeps that beam's; each
// further one takes over the page (and those behind it) of a beam that no place
// continues, of which there are as many, and the rows that p's last page holds are
// copied there.  So nothing is allocated, as little as can be is copied, and no page
// is both read and written.  Every workgroup works the exchange out for itself,
// a lane to a place; one of each group and place writes its table, the others copy one
// place's rows of one layer, eight units a thread in flight.  Bound by the chain of
// dependent loads (parents, table, row) and HBM: 32 groups of 8 beams in 12 layers of 8
// bits, 47 MB, 12.3 us; four beams of one layer 3.4.
constexpr int kReorderThreads = 256;
constexpr int kCopyBatch = 8;

template <bool Q8>
__global__ __launch_bounds__(kReorderThreads) void reorder_kernel(ReorderArgs a) {
    const int tid = threadIdx.x, lane = tid & 63, g = blockIdx.x, w = a.beams;
    const int layer = static_cast<int>(blockIdx.y) - 1, place = blockIdx.z;
    const int64_t seq0 = static_cast<int64_t>(g) * w;
    const bool here = lane < w;
    int parent = here ? a.parents[seq0 + lane] : -1;
    const int mine = here ? a.kv_len[seq0 + lane] : 0, len = __builtin_amdgcn_readfirstlane(mine);
    const bool report = layer < 0 && place == 0 && tid < 64;
    bool known = parent >= 0 && parent < w;
    const bool bad_len = __any(here && (mine != len || len < 0));
    dev::flag_if(report && here && !known && parent != -1, a.err, kErrDraft);
    dev::flag_if(report && bad_len, a.err, kErrSeq);
    if (bad_len) {                                        // the group stays as it is
        parent = lane;
        known = here;
    }
    uint64_t used = 0;
    bool extra = here && !known;
    for (int j = 0; j < w; ++j) {
        const int p = __builtin_amdgcn_readlane(parent, j);
        if (p < 0 || p >= w) continue;
        if (known && p == parent && j < lane) extra = true;
        used |= 1ull << p;
    }
    const uint64_t extras = __ballot(extra);
    const int rank = __popcll(extras & ((1ull << lane) - 1));
    int donor = parent, seen = 0;
    for (int p = 0; p < w; ++p)                           // the rank-th beam that nobody continues
        if (!((used >> p) & 1)) {
            if (extra && seen == rank) donor = p;
            ++seen;
        }
    if (here && !known) parent = donor;                   // the place keeps a beam that is left over
    const int shift = a.cache.page_shift, whole = len >> shift, part = len & ((1 << shift) - 1);
    if (layer < 0) {
        // Tables: place by place, the columns before the last page from the parent.
        const int from = __builtin_amdgcn_readlane(parent, place), to = __builtin_amdgcn_readlane(donor, place);
        const int32_t *head = a.cache.table + (seq0 + from) * a.cache.table_stride, *tail = a.cache.table + (seq0 + to) * a.cache.table_stride;
        int32_t *out = a.out_table + (seq0 + place) * a.out_stride;
        for (int c = tid; c < a.cache.table_cols; c += kReorderThreads) out[c] = c < whole && !bad_len ? head[c] : tail[c];
        return;
    }
    const int from = __builtin_amdgcn_readlane(parent, place), to = __builtin_amdgcn_readlane(donor, place);
    if (from == to || part == 0) return;
    int src = -1, dst = -1;
    if (whole < a.cache.table_cols) {
        src = a.cache.table[(seq0 + from) * a.cache.table_stride + whole];
        dst = a.cache.table[(seq0 + to) * a.cache.table_stride + whole];
    }
    if (src < 0 || src >= a.cache.n_pages || dst < 0 || dst >= a.cache.n_pages) {
        dev::flag_if(tid == 0 && layer == 0, a.err, kErrPage);
        return;
    }
    uint8_t *base = a.cache.base + layer * a.layer_bytes;
    const u32x4 *x = reinterpret_cast<const u32x4 *>(base + src * a.cache.page_bytes);
    u32x4 *y = reinterpret_cast<u32x4 *>(base + dst * a.cache.page_bytes);
    const int units = part * kRowUnits<Q8>;
    for (int u0 = tid; u0 < units; u0 += kCopyBatch * kReorderThreads) {
        u32x4 v[kCopyBatch];
#pragma unroll
        for (int i = 0; i < kCopyBatch; ++i)
            if (u0 + i * kReorderThreads < units) v[i] = x[u0 + i * kReorderThreads];
#pragma unroll
        for (int i = 0; i < kCopyBatch; ++i)
            if (u0 + i * kReorderThreads < units) y[u0 + i * kReorderThreads] = v[i];
    }
}

}  // namespace

hipError_t launch_append(const AppendArgs &a, bool bf16, bool cache8, hipStream_t s) {
    launch(cache8 ? (bf16 ? append_kernel<true, true> : append_kernel<false, true>) : (bf16 ? append_kernel<true, false> : append_kernel<false, false>),
           static_cast<unsigned>(a.n_tok), kAppendThreads, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_keep(const KeepArgs &a, bool cache8, hipStream_t s) {
    const int64_t units = static_cast<int64_t>(a.n_layers) * a.n_seq * (cache8 ? kRowUnits<true> : kRowUnits<false>);
    const int64_t blocks = (units + kKeepThreads - 1) / kKeepThreads;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    launch(cache8 ? keep_kernel<true> : keep_kernel<false>, static_cast<unsigned>(blocks), kKeepThreads, 0, s, a, units);
    return hipGetLastError();
}

hipError_t launch_read(const ReadArgs &a, bool bf16, bool cache8, hipStream_t s) {
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(a.n_rows) + kReadRows - 1) / kReadRows);
    const bool stream = static_cast<int64_t>(a.n_rows) * kRowBytes > kStreamBytes;
    launch(cache8 ? (bf16 ? (stream ? read_kernel<true, true, true> : read_kernel<true, true, false>)
                          : (stream ? read_kernel<false, true, true> : read_kernel<false, true, false>))
                  : (stream ? read_kernel<true, false, true> : read_kernel<true, false, false>),
           blocks, kReadThreads, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_reorder(const ReorderArgs &a, bool cache8, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.n_groups), static_cast<unsigned>(a.n_layers) + 1, static_cast<unsigned>(a.beams));
    launch(cache8 ? reorder_kernel<true> : reorder_kernel<false>, grid, kReorderThreads, 0, s, a);
    return hipGetLastError();
}

}  // namespace coli
