// latent_decode.hip -- absorbed latent attention of single, chained or
// tree-drafted tokens over the paged latent cache.
//
// Every head of a token attends to the same 576 cached values per key (512
// latent ones that are key and value, 64 rotary ones that are key only):
//   s_j = scale (q_lat . c_j + q_pe . r_j),  o = sum_j softmax(s)_j c_j,
// so the (token, head) pairs of a sequence are rows of one product and a key
// is read once for 64 of them.  One workgroup of eight waves has a CU to
// itself and takes 64 rows and a run of keys in steps of 32, with the running
// maximum and sum of the softmax.  Each SIMD holds a wave of either kind:
//   - a scoring wave computes S^T = K Q^T of step t, 16 keys x 32 rows, with its
//     rows' queries in 144 registers, and writes the probabilities to LDS, in the
//     16 bits that the second product takes (their fp32 sum is taken before;
//     bf16 outputs are off by 2.0e-3 of their size, 1.7e-3 by their own rounding);
//   - a summing wave computes O^T += V^T P^T of step t - 1, 64 rows x 128 latent
//     columns in 128 registers, reading V^T with transposed LDS reads, and
//     copies the keys of step t + 2 (36 KB a step, a ring of four) from the
//     cache straight into LDS.
// The two meet at one barrier a step.  Between barriers each has latencies
// that it cannot hide by itself (its first LDS reads, the exponentials, the
// issue of the copies); the products of the other fill them.  One kind of
// wave doing both in turn, at one wave per SIMD, took 1.37 us a step against
// the 0.45 us of its products.
// Splitting the keys of the first product and the columns of the second means
// that each wave reads half of K or a quarter of V from LDS; with rows alone
// split every wave would read all of both.
//
// A sequence's keys are cut into pieces so that every CU has one (the plan);
// pieces leave unnormalised sums, maxima and fp32 partial outputs, which
// join_kernel combines.
//
// Measured.  64 tokens of sequences up to 12k, 64 heads, bf16: 67 us and 10 for the
// join, 352 MB, 5.3 TB/s in the first: bound by HBM.  Four chains of four tokens up
// to 128k, 16 heads, f16: 92 and 13 us, 535 MB, 5.8 TB/s.  16 trees of 25 nodes up
// to 5k, 64 heads, bf16: 149 us, 960 TFLOP/s against 1223 of a large library
// product; the matrix pipes are busy 43% of the cycles at 2.1 GHz, the product's 70%
// at 1.5 to 1.9.  One token, 4k, 64 heads: 11.5 and 5.7 us, a chain of latencies (the
// item, its queries, page numbers, keys, four steps, partial results).
//
// Over an 8-bit cache the summing waves also convert (Source8).  64 tokens of
// sequences up to 12k, 64 heads, f16: 69 us and 9.4 for the join, 204 MB; one token, 4k:
// 12.7 and 5.2.  Bound by its steps, 1.3 us each: 64 tokens of 8192 take 110 us, 111 from
// 16 bits; 84 without the copies, and resident 100, 81 without the conversion.
// A unit of 32 rows or fewer does half of the products (16 heads, 64 tokens of 8192: 8
// bits 109 -> 94 us, 16 bits 112 -> 108) and leaves half a piece (16 heads, 32 tokens of
// 600 to 12000: 48.9 -> 45.5).
#include "dev_attn.h"

namespace coli {
namespace {

using dev::f32x16;
using dev::f32x4;
using dev::u32x2;
using dev::u32x4;

constexpr int kStepKeys = 32;
constexpr int kBlocks = kCacheRow / 64;                  // 64-column blocks of a cached row: 8 latent, 1 rotary
constexpr int kLatentBlocks = kLatent / 64;
constexpr int kBlockBytes = kStepKeys * 128;
constexpr int kStepBytes = kBlocks * kBlockBytes;        // 36 KB
// Steps in LDS.  Of a 16-bit cache: one that is summed, one that is scored and two on
// their way.  Those of an 8-bit cache on their way lie apart, as they come; a third place
// is being written.
template <bool Q8>
constexpr int kRing = Q8 ? 3 : 4;
constexpr int kRawBytes = kStepKeys / 4 * kRow8Bytes;    // a summing wave's share of a step on its way
constexpr int kWeightBytes = 2 * kTileRows * 64;
template <bool Q8>
constexpr int kKeyBytes = kRing<Q8> * kStepBytes;
constexpr int kDepth = kCacheRow / 32;                   // K steps of the first product
// The running maximum of a row moves only when a step exceeds it by more than
// 2^kSlack: the accumulator is then rarely rescaled, and probabilities stay
// below 2^kSlack, far inside the range of both 16-bit types and of the sums.
constexpr float kSlack = 8.0f;
constexpr int kKeyAhead = 6;                             // LDS reads in flight ahead of the products that use them
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

// Probabilities of a step: 64 rows of 32 keys, 64 bytes a row; the XOR spreads
// 16 rows read at one 16-byte unit over all banks.
__device__ __forceinline__ int weight_unit(int r, int q) { return r * 64 + ((q ^ ((r >> 2) & 3)) << 4); }

// Which of the 64 keys from key0 on a row sees, as bits.  Rows of a chain see keys up to
// their own position; rows of a tree see the context and the nodes of their
// ancestor bits.
__device__ __forceinline__ uint64_t below(int c) { return c >= 64 ? ~0ull : c <= 0 ? 0ull : (1ull << c) - 1; }
__device__ __forceinline__ uint64_t seen_keys(const DecodeArgs &a, const DecodeItem &it, int node, int key0) {
    const int ctx = it.len - it.n;
    if (!a.mask) return below(ctx + node + 1 - key0);
    const uint64_t *m = a.mask + static_cast<int64_t>(it.q0 + node) * a.mask_words;
    const int d = key0 - ctx;                            // node index of the first key
    uint64_t v;
    if (d <= -64) {
        v = ~0ull;
    } else if (d < 0) {
        v = (m[0] << -d) | below(-d);
    } else {
        const int w = d >> 6, s = d & 63;
        v = w < a.mask_words ? m[w] >> s : 0ull;
        if (s && w + 1 < a.mask_words) v |= m[w + 1] << (64 - s);
    }
    return v & below(it.len - key0);
}

constexpr int kThreads = 512;

// What both kinds of wave know of an item.
struct Shared {
    uint8_t *kv, *p;                   // [kRing] steps of keys; [2] steps of probabilities
    uint8_t *raw;                      // of an 8-bit cache: [4 waves][2] shares of steps on their way
    float *red, *fac, *sum;            // [2][2][64] maxima by step parity and key half; [64]; [2][64]
    int *raise, *bad;                  // [3] by step; one flag
    int t0, t1, open;                  // steps; keys below `open` are seen by every row
    template <bool Q8>
    __device__ uint8_t *ring(int t) const { return kv + (Q8 ? (t - t0) % kRing<Q8> : (t - t0) & (kRing<Q8> - 1)) * kStepBytes; }
    __device__ uint8_t *weights(int t) const { return p + (t & 1) * (kTileRows * 64); }
    __device__ float *maxima(int t, int half) const { return red + ((t & 1) * 2 + half) * kTileRows; }
};

// In the careful pass, values that are not finite are taken as zero in the steps
// that hide keys from some row: such keys hold what other branches left there,
// their weight is zero, and zero times inf or NaN must not reach a row that does
// not see them.  spoil_seen() then sees to the rows that do.
template <bool BF, bool Q8>
__device__ __forceinline__ void clean(const Shared &sh, int t) {
    dev::lds_barrier();                                  // every wave has read the step's keys; the copies in flight are of other steps
    u32x4 *v = reinterpret_cast<u32x4 *>(sh.ring<Q8>(t));
    for (int i = threadIdx.x; i < kLatentBlocks * kBlockBytes / 16; i += kThreads) {
        u32x4 w = v[i];
#pragma unroll
        for (int d = 0; d < 4; ++d) w[d] &= ~dev::nonfinite_halves<BF>(w[d]);
        v[i] = w;
    }
    dev::lds_barrier();
}

// A summing wave's share of an 8-bit cache's steps: of each step keys 8 wave .. + 7, whose
// bytes it copies into LDS two steps ahead, as they lie in memory, and then writes into
// the ring as the 16-bit values that they stand for: the scoring waves work as on a
// 16-bit cache.  (Every stored value is one of the 16-bit type: the scales are powers of
// two within its range.)  A wave waits for its own copies alone.
// 64 tokens of 8192, 64 heads: 110 us.  With the bytes in registers instead of LDS until
// their step 67 spill; with all eight waves converting four keys 112 to 116, with scoring
// waves converting what they score 114, with values read a step ahead and three steps on
// their way 110 to 114.
template <bool ONCE>
struct Source8 {
    static constexpr int kUnits = kRow8Bytes / 16, kKeys = 8, kCopies = (kKeys * kUnits + 63) / 64;
    const uint8_t *base, *raw;
    const int32_t *table;
    int64_t page_bytes;
    uint32_t raw_lds;
    int shift, cols, n_pages, len, t0, last, key0;
    bool bad = false;
    int page = 0;                      // of the keys of the step that is copied next
    // Of a step between its wait and its writing.
    u32x2 q[8];
    u32x4 pe;
    uint32_t by;

    __device__ __forceinline__ Source8(const DecodeArgs &a, const DecodeItem &it, const Shared &sh, uint32_t lds)
        : base(a.cache.base), raw(sh.raw + (dev::wave_id() & 3) * 2 * kRawBytes), table(a.cache.table + it.seq * a.cache.table_stride),
          page_bytes(a.cache.page_bytes), raw_lds(lds + (dev::wave_id() & 3) * 2 * kRawBytes), shift(a.cache.page_shift), cols(a.cache.table_cols),
          n_pages(a.cache.n_pages), len(it.len), t0(sh.t0), last(sh.t1 - 1), key0(kKeys * (dev::wave_id() & 3)) {}
    // Past the end the last step is copied again, and keys past the last one are that one.
    __device__ __forceinline__ int position(int t) const { return min(min(t, last) * kStepKeys + key0, len - 1); }
    // Pages of eight rows or more hold all of the wave's keys; their number is read by the
    // scalar unit a step ahead.
    __device__ __forceinline__ void ask(int t) { page = dev::ld_uniform(table + min(position(t) >> shift, max(cols, 1) - 1)); }
    __device__ __forceinline__ const uint8_t *row_at(int pos, int page) {
        const bool off = page < 0 || page >= n_pages || pos >> shift >= cols;
        bad = bad || off;
        return base + (off ? 0 : page) * page_bytes + (pos & ((1 << shift) - 1)) * kRow8Bytes;
    }
    static __device__ __forceinline__ void copy16(const uint8_t *src, uint32_t dst) {
        if constexpr (ONCE) dev::copy16_to_lds_once(src, dst);
        else dev::copy16_to_lds_free(src, dst);
    }
    __device__ __forceinline__ void copy(int t) {
        const int lane = threadIdx.x & 63, pos = position(t), most = len - 1 - pos;
        const uint32_t dst = raw_lds + ((t - t0) & 1) * kRawBytes;
        if (shift >= 3 && most >= kKeys - 1) {
            const uint8_t *r = row_at(pos, page) + 16 * lane;
#pragma unroll
            for (int i = 0; i < kKeys * kUnits / 64; ++i) copy16(r + 1024 * i, dst + 1024 * i);
            if (lane < kKeys * kUnits % 64) copy16(r + 1024 * (kCopies - 1), dst + 1024 * (kCopies - 1));
        } else {
            // The last keys, or small pages: each lane finds its key's row.  (Vector loads of
            // the table wait for the copies in flight, no more.)
#pragma unroll 1
            for (int i = 0; i < kCopies; ++i) {
                const int u = 64 * i + lane, k = u / kUnits, p = pos + min(k, most), at = p >> shift;
                if (u < kKeys * kUnits) {
                    int page = table[min(at, max(cols, 1) - 1)];
                    asm volatile("" : "+v"(page));
                    const bool off = page < 0 || page >= n_pages || at >= cols;
                    bad = bad || off;
                    copy16(base + (off ? 0 : page) * page_bytes + (p & ((1 << shift) - 1)) * kRow8Bytes + 16 * (u - k * kUnits), dst + 1024 * i);
                }
            }
        }
    }
    // Step t into registers, and step t + 2 on its way in its place.  Lane L holds 64 values
    // of key L / 8, 16 of each 128 columns from 16 (L % 8) on, the scales' bytes, and 8 rotary
    // values.  Of 16 values the upper four lanes of a key take the upper half first:
    // they lie in the same places of another block, and are written at the same time.
    __device__ __forceinline__ void fetch(int t) {
        const int lane = threadIdx.x & 63, c = lane & 7;
        const uint8_t *from = raw + ((t - t0) & 1) * kRawBytes + (lane >> 3) * kRow8Bytes;
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCopies) : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) q[2 * j + h] = *reinterpret_cast<const u32x2 *>(from + 128 * j + 16 * c + 8 * (h ^ (c >> 2)));
        by = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) by |= static_cast<uint32_t>(from[kRow8Scales + 4 * j + (c >> 1)]) << (8 * j);
        pe = *reinterpret_cast<const u32x4 *>(from + kRow8Rope + 16 * c);
    }
    __device__ __forceinline__ void copy_next(int t) {
        asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(q[0]), "+v"(q[1]), "+v"(q[2]), "+v"(q[3]), "+v"(q[4]), "+v"(q[5]), "+v"(q[6]), "+v"(q[7]), "+v"(pe), "+v"(by)::"memory");
        copy(t + 2);
    }
    template <bool BF>
    __device__ __forceinline__ void write(uint8_t *place, int j) const {
        const int lane = threadIdx.x & 63, c = lane & 7, r = key0 + (lane >> 3);
        const float f = __uint_as_float(j == 0 ? by << 23 : by >> (8 * j) << 23);   // of a scale the conversion sees the exponent bits alone
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<u32x4 *>(place + (2 * j + (c >> 2)) * kBlockBytes + dev::tile_unit(r, 2 * (c & 3) + (h ^ (c >> 2)))) =
                u32x4{dev::of_fp8<BF, false>(q[2 * j + h][0], f), dev::of_fp8<BF, true>(q[2 * j + h][0], f), dev::of_fp8<BF, false>(q[2 * j + h][1], f),
                      dev::of_fp8<BF, true>(q[2 * j + h][1], f)};
        if (j == 3) *reinterpret_cast<u32x4 *>(place + kLatentBlocks * kBlockBytes + dev::tile_unit(r, c)) = pe;
    }
    template <bool BF>
    __device__ __forceinline__ void pass_on(int t, uint8_t *place) {
        fetch(t);
        copy_next(t);
#pragma unroll
        for (int j = 0; j < 4; ++j) write<BF>(place, j);
    }
};

// The scoring waves' part of an item: wave (wm, wk) scores keys 16 wk .. + 15 of
// each step for rows 32 wm .. + 31; lane L owns rows row and row + 16, row =
// 32 wm + L % 16.  Leaves the running maxima in m.
template <bool BF, bool Q8>
__device__ __forceinline__ void score_item(const DecodeArgs &a, const DecodeItem &it, const Shared &sh, int rows, bool careful,
                                           float (&m)[2]) {
    const int lane = threadIdx.x & 63, wave = dev::wave_id();
    const int wm = wave & 1, wk = (wave >> 1) & 1, l15 = lane & 15, lq = lane >> 4;
    const int row = 32 * wm + l15;
    const float c = a.scale * kLog2e;
    int node[2];
    u32x4 q[kDepth][2];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) node[rb] = (it.row0 + min(row + 16 * rb, rows - 1)) / a.n_heads;
    if (sh.t0 < sh.t1) {
        // The queries come by way of the ring's last two places, each row once and
        // whole, which leaves the keys' copies room: loaded by each wave as
        // its products take them, they let the first step begin 11400 clocks after
        // the item, so 3900 (one token, 4096 keys 19.9 -> 16.9 us).
        const int r = 8 * wave + (lane >> 3), unit = ((lane & 7) ^ dev::tile_swz(r)) << 4;
        const uint32_t at = dev::lds_address(sh.kv) + (kRing<Q8> - 2) * kStepBytes + wave * 1024;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int rr = it.row0 + min(r + 32 * h, rows - 1), n = rr / a.n_heads, head = rr - n * a.n_heads;
            const int64_t tok = it.q0 + n;
            const uint8_t *ql = a.q_lat + (tok * a.ql_tok + head * a.ql_head) * 2 + unit;
            const uint8_t *qp = a.q_pe + (tok * a.qp_tok + head * a.qp_head) * 2 + unit;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                dev::copy16_to_lds_free(b < kLatentBlocks ? ql + 128 * b : qp, at + h * kStepBytes + b * kBlockBytes);
        }
        dev::copy_barrier();
        const uint8_t *mine = sh.kv + (kRing<Q8> - 2 + wm) * kStepBytes;
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
#pragma unroll
            for (int rb = 0; rb < 2; ++rb)
                q[k][rb] = *reinterpret_cast<const u32x4 *>(mine + (k >> 1) * kBlockBytes + dev::tile_unit(l15 + 16 * rb, 4 * (k & 1) + lq));
    }
    __builtin_amdgcn_s_setprio(2);   // the step waits for these waves: the summing ones fill what they leave
    m[0] = m[1] = -__builtin_inff();
    float l[2] = {0.0f, 0.0f};
    f32x4 s[2] = {}, s_prev[2] = {};
    float sum_prev[2] = {0.0f, 0.0f};
    // With 32 rows or fewer two of the waves have none, and only keep up with the barriers.
    const bool idle = 32 * wm >= rows;
    auto score = [&](int t) {
        if (idle) return;
        const uint8_t *kr = sh.ring<Q8>(t) + 16 * wk * 128;
        auto key = [&](int k) {
            return *reinterpret_cast<const u32x4 *>(kr + (k >> 1) * kBlockBytes + dev::tile_unit(l15, 4 * (k & 1) + lq));
        };
        u32x4 kf[kKeyAhead];
#pragma unroll
        for (int k = 0; k < kKeyAhead; ++k) kf[k] = key(k);
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) s[rb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
#pragma unroll
            for (int rb = 0; rb < 2; ++rb) s[rb] = dev::mma16<BF>(kf[k % kKeyAhead], q[k][rb], s[rb]);
            if (k + kKeyAhead < kDepth) kf[k % kKeyAhead] = key(k + kKeyAhead);
        }
        dev::pipeline<kDepth, 2, 1, kKeyAhead>();
        __builtin_amdgcn_sched_barrier(0);
        if ((t + 1) * kStepKeys > sh.open) {
#pragma unroll
            for (int rb = 0; rb < 2; ++rb) {
                const uint32_t seen = static_cast<uint32_t>(seen_keys(a, it, node[rb], t * kStepKeys)) >> (16 * wk + 4 * lq);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!((seen >> i) & 1)) s[rb][i] = -__builtin_inff();
            }
        }
    };
    // What the fast path needs of the running maxima: the score that calls for
    // a new one, and the exponent's offset.
    float limit[2], offset[2];
    auto set_limits = [&]() {
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
            limit[rb] = (m[rb] + kSlack) / c;
            offset[rb] = m[rb] == -__builtin_inff() ? 0.0f : -m[rb];
        }
    };
    auto lane_max = [&](const f32x4 &v) { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); };
    auto post_max = [&](int t, const f32x4 (&v)[2]) {
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
            const float x = dev::max_halves(dev::max_quarters(lane_max(v[rb])));
            if (lq == 0) sh.maxima(t, wk)[row + 16 * rb] = x;
        }
    };
    // Probabilities of scores v against the running maxima; the lane's part of
    // the row sums.
    auto weigh = [&](int t, const f32x4 (&v)[2], float (&sum)[2]) {
        if (idle) return;
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[rb][i], c, offset[rb]));
            sum[rb] = (p[0] + p[1]) + (p[2] + p[3]);
            *reinterpret_cast<u32x2 *>(sh.weights(t) + weight_unit(row + 16 * rb, 2 * wk + (lq >> 1)) + 8 * (lq & 1)) =
                u32x2{dev::pack2<BF>(p[0], p[1]), dev::pack2<BF>(p[2], p[3])};
        }
    };
    // New maxima from both key halves of step t, and the factors of what was
    // summed before it.
    auto take_max = [&](int t, float slack) {
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
            const int r = row + 16 * rb;
            const float tm = fmaxf(sh.maxima(t, 0)[r], sh.maxima(t, 1)[r]) * c;
            const float m1 = tm > m[rb] + slack ? tm : m[rb];
            const float fac = m1 == m[rb] ? 1.0f : __builtin_amdgcn_exp2f(m[rb] - m1);
            m[rb] = m1;
            l[rb] *= fac;
            if (wk == 0 && lq == 0) sh.fac[r] = fac;
        }
        set_limits();
    };
    // After the barrier behind step t: where a row exceeded its maximum by
    // more than the slack, the maxima are exchanged and the step is weighed
    // again.
    auto settle = [&](int t, int raise) {
        if (__builtin_amdgcn_readfirstlane(raise)) {
            post_max(t, s_prev);
            dev::lds_barrier();
            take_max(t, kSlack);
            weigh(t, s_prev, sum_prev);
            dev::lds_barrier();
        }
        l[0] += sum_prev[0];
        l[1] += sum_prev[1];
        if (careful && (t + 1) * kStepKeys > sh.open) clean<BF, Q8>(sh, t);
    };
    if (sh.t0 < sh.t1) {
        // First step: its maxima are exchanged before it is weighed.
        dev::lds_barrier();
        score(sh.t0);
        post_max(sh.t0, s);
        dev::lds_barrier();
        take_max(sh.t0, 0.0f);
        weigh(sh.t0, s, sum_prev);
        s_prev[0] = s[0];
        s_prev[1] = s[1];
        for (int t = sh.t0 + 1; t < sh.t1; ++t) {
            dev::lds_barrier();
            const int raise = sh.raise[(t - 1 - sh.t0) % 3];
            if (threadIdx.x == 0) sh.raise[(t + 1 - sh.t0) % 3] = 0;
            score(t);
            settle(t - 1, raise);
            weigh(t, s, sum_prev);
            if (__any(lane_max(s[0]) > limit[0] || lane_max(s[1]) > limit[1])) sh.raise[(t - sh.t0) % 3] = 1;
            s_prev[0] = s[0];
            s_prev[1] = s[1];
        }
        dev::lds_barrier();
        settle(sh.t1 - 1, sh.raise[(sh.t1 - 1 - sh.t0) % 3]);
    }
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
        const float sum = dev::sum_halves(dev::sum_quarters(l[rb]));
        if (lq == 0) sh.sum[wk * kTileRows + row + 16 * rb] = sum;
    }
}

// The summing waves' part: wave w copies keys 8 w .. + 7 of each step and sums
// columns 128 w .. + 127 for all rows.
template <bool BF, bool ONCE, bool Q8>
__device__ __forceinline__ void sum_item(const DecodeArgs &a, const DecodeItem &it, const Shared &sh, uint32_t kv_lds, uint32_t raw_lds, int rows, bool careful,
                                         bool &bad_page, f32x16 (&acc)[4][2]) {
    const int lane = threadIdx.x & 63, wave = dev::wave_id() & 3, l31 = lane & 31, lh = lane >> 5;
#pragma unroll
    for (int cb = 0; cb < 4; ++cb)
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[cb][rb][i] = 0.0f;
    if (sh.t0 >= sh.t1) return;
    // Each lane copies one 16-byte unit of every block of one key.  Pages of
    // eight rows or more hold all of a wave's keys: the page number is then the
    // wave's, read by the scalar unit a step ahead (a vector load in flight
    // would make its use wait for the copies issued before it).
    const int cr = 8 * wave + (lane >> 3);
    const int cu = ((lane & 7) ^ dev::tile_swz(cr)) << 4;
    const int32_t *table = a.cache.table + it.seq * a.cache.table_stride;
    const int shift = a.cache.page_shift, cols = a.cache.table_cols, last = sh.t1 - 1;
    const bool wide = shift >= 3;
    auto page_of = [&](int t) {
        const int pos = min(min(t, last) * kStepKeys + 8 * wave, it.len - 1);
        return dev::ld_uniform(table + min(pos >> shift, max(cols, 1) - 1));
    };
    struct Copy {
        const uint8_t *src;
        uint32_t dst;
    };
    auto aim = [&](int t, int wave_page) {
        t = min(t, last);                                // past the end the last step is copied again
        const int pos = min(t * kStepKeys + cr, it.len - 1), at = pos >> shift;
        int page = wave_page;
        if (!wide) {
            page = table[min(at, max(cols, 1) - 1)];
            asm volatile("" : "+v"(page));               // waited for here, not (with the copies) where the paths join
        }
        if (page < 0 || page >= a.cache.n_pages || at >= cols) {
            bad_page = true;
            page = 0;
        }
        return Copy{a.cache.base + page * a.cache.page_bytes + (pos & ((1 << shift) - 1)) * kRowBytes + cu,
                    kv_lds + ((t - sh.t0) & (kRing<false> - 1)) * kStepBytes + wave * 1024};
    };
    auto copy = [&](const Copy &x, int b) {
        if constexpr (ONCE) dev::copy16_to_lds_once(x.src + b * 128, x.dst + b * kBlockBytes);
        else dev::copy16_to_lds_free(x.src + b * 128, x.dst + b * kBlockBytes);
    };
    auto copy_all = [&](const Copy &x) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) copy(x, b);
    };
    // Sums step t.  In the loop the copies `now` (of step t + 3) are issued
    // between the products, and what the next ones need is computed there: four
    // waves' copies keep the CU's address unit busy for about 900 clocks, nearly
    // as long as both kinds' products take.
    const int kr0 = 8 * lh + ((lane >> 2) & 3);
    Source8<ONCE> src(a, it, sh, raw_lds);
    auto step = [&](int t, bool more, Copy &now, int &page) {
        const int raise = sh.raise[(t - sh.t0) % 3];
        const uint8_t *vr = sh.ring<Q8>(t) + 2 * wave * kBlockBytes + 8 * (lane & 1);
        const uint8_t *pr = sh.weights(t);
        u32x4 pf[2][2], vf[2][4];
        auto read_weights = [&]() {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int rb = 0; rb < 2; ++rb) pf[k][rb] = *reinterpret_cast<const u32x4 *>(pr + weight_unit(32 * rb + l31, 2 * k + lh));
        };
        auto read_values = [&]() {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) {
                    const uint8_t *blk = vr + (cb >> 1) * kBlockBytes + 16 * k * 128;
                    const int unit = 4 * (cb & 1) + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
                    const u32x2 a0 = dev::read_tr(blk + dev::tile_unit(kr0, unit));
                    const u32x2 a1 = dev::read_tr(blk + dev::tile_unit(kr0 + 4, unit));
                    vf[k][cb] = u32x4{a0[0], a0[1], a1[0], a1[1]};
                }
        };
        read_weights();
        read_values();
        __builtin_amdgcn_sched_barrier(0);
        if (__builtin_amdgcn_readfirstlane(raise)) {
            dev::lds_barrier();                          // maxima
            dev::lds_barrier();                          // weights and factors
            read_weights();
            const float f0 = sh.fac[l31], f1 = sh.fac[32 + l31];
#pragma unroll
            for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    acc[cb][0][i] *= f0;
                    acc[cb][1][i] *= f1;
                }
        }
        if (careful && (t + 1) * kStepKeys > sh.open) {
            clean<BF, Q8>(sh, t);
            read_values();
        }
        Copy next = now;
        if (Q8 && more) src.ask(t + 4);
        if (!Q8 && more) copy(now, 0);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int rb = 0; rb < 2; ++rb)
                    if (rb == 0 || rows > 32) acc[cb][rb] = dev::mma<BF>(vf[k][cb], pf[k][rb], acc[cb][rb]);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (Q8) {
                    if (more && k == 0 && cb == 0) src.fetch(t + 2);
                    if (more && k == 0 && cb == 2) src.copy_next(t + 2);
                    if (more && k == 1) src.template write<BF>(sh.ring<Q8>(t + 2), cb);
                } else {
                    if (more) copy(now, 1 + 4 * k + cb);
                    if (more && k == 1 && cb == 1) {
                        next = aim(t + 4, page);
                        page = page_of(t + 5);
                    }
                }
            }
        now = next;
    };

    Copy now{};
    int page = 0;
    if constexpr (Q8) {
        src.ask(sh.t0);
        src.copy(sh.t0);
        src.ask(sh.t0 + 1);
        src.copy(sh.t0 + 1);
        src.ask(sh.t0 + 2);
        dev::lds_barrier();                              // the queries have landed
        src.template pass_on<BF>(sh.t0, sh.ring<Q8>(sh.t0));
        src.ask(sh.t0 + 3);
        dev::lds_barrier();                              // step t0 has been written, and the queries have been read
        src.template pass_on<BF>(sh.t0 + 1, sh.ring<Q8>(sh.t0 + 1));
        dev::lds_barrier();                              // the first maxima
        for (int t = sh.t0 + 1; t < sh.t1; ++t) {
            dev::lds_barrier();
            step(t - 1, true, now, page);
        }
        dev::copy_barrier();                             // what was copied past the end has landed too
        bad_page = bad_page || src.bad;
    } else {
        const int pg0 = page_of(sh.t0), pg1 = page_of(sh.t0 + 1), pg2 = page_of(sh.t0 + 2), pg3 = page_of(sh.t0 + 3);
        page = page_of(sh.t0 + 4);
        copy_all(aim(sh.t0, pg0));
        copy_all(aim(sh.t0 + 1, pg1));
        now = aim(sh.t0 + 2, pg2);
        dev::lds_barrier();                              // the queries have landed
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kBlocks) : "memory");
        dev::lds_barrier();                              // step t0 has landed, and the queries have been read
        copy_all(now);
        now = aim(sh.t0 + 3, pg3);
        dev::lds_barrier();                              // the first maxima
        for (int t = sh.t0 + 1; t < sh.t1; ++t) {
            // Step t has landed when only the copies of step t + 1 are in flight.
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kBlocks) : "memory");
            dev::lds_barrier();
            step(t - 1, true, now, page);
        }
        dev::copy_barrier();
    }
    step(last, false, now, page);
    float z = 0.0f;
#pragma unroll
    for (int cb = 0; cb < 4; ++cb)
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
            for (int i = 0; i < 16; ++i) z = __builtin_fmaf(acc[cb][rb][i], 0.0f, z);
    if (__any(z != 0.0f)) *sh.bad = 1;
}

// After the careful pass: outputs whose value is not finite in a key that their row
// sees, in the steps that were cleaned, become NaN, as they do by themselves in
// the other steps.  (An infinite latent is part of the key too: the row's score is
// then NaN or +inf and the whole row NaN, or it is -inf and the output 0 * inf.)
// The keys are read from the cache again, eight at a time: this is rare, and a count
// of them beside the products, in the registers that those leave, spills 673.
template <bool BF, bool Q8>
__device__ __forceinline__ void spoil_seen(const DecodeArgs &a, const DecodeItem &it, const Shared &sh, int rows, f32x16 (&acc)[4][2]) {
    const int lane = threadIdx.x & 63, wave = dev::wave_id() & 3, l31 = lane & 31, lh = lane >> 5;
    const int32_t *table = a.cache.table + it.seq * a.cache.table_stride;
    const int shift = a.cache.page_shift, cols = a.cache.table_cols;
    const int node0 = (it.row0 + min(l31, rows - 1)) / a.n_heads, node1 = (it.row0 + min(32 + l31, rows - 1)) / a.n_heads;
    constexpr int kBatch = 8;
    uint64_t even[2] = {0, 0}, odd[2] = {0, 0};          // of the lane's two rows: columns 128 wave + 2 bit (and + 1) to spoil
#pragma unroll 1
    for (int key = max(sh.t0, max(sh.open, 0) / kStepKeys) * kStepKeys; key < min(sh.t1 * kStepKeys, it.len); key += kBatch) {
        uint32_t off[kBatch], any = 0;                   // of values 128 wave + 2 lane and the next
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int pos = min(key + j, it.len - 1), at = pos >> shift;
            int page = dev::ld_uniform(table + min(at, max(cols, 1) - 1));
            if (page < 0 || page >= a.cache.n_pages || at >= cols) page = 0;   // flagged where it was copied
            const uint8_t *row = a.cache.base + page * a.cache.page_bytes + (pos & ((1 << shift) - 1)) * (Q8 ? kRow8Bytes : kRowBytes);
            if constexpr (Q8)
                off[j] = dev::of_fp8<BF, false>(*reinterpret_cast<const uint16_t *>(row + 128 * wave + 2 * lane),
                                                __uint_as_float(static_cast<uint32_t>(row[kRow8Scales + 4 * wave + (lane >> 4)]) << 23));
            else
                off[j] = *reinterpret_cast<const uint32_t *>(row + 256 * wave + 4 * lane);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            off[j] = dev::nonfinite_halves<BF>(off[j]);
            any |= off[j];
        }
        if (!__any(any != 0)) continue;
        const uint64_t seen0 = seen_keys(a, it, node0, key), seen1 = seen_keys(a, it, node1, key);   // none past the last key
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint64_t e = __ballot(off[j] & 0xFFFFu), o = __ballot(off[j] >> 16);
            if ((seen0 >> j) & 1) {
                even[0] |= e;
                odd[0] |= o;
            }
            if ((seen1 >> j) & 1) {
                even[1] |= e;
                odd[1] |= o;
            }
        }
    }
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
        even[rb] >>= 2 * lh;
        odd[rb] >>= 2 * lh;
#pragma unroll
        for (int cb = 0; cb < 4; ++cb)
#pragma unroll
            for (int i = 0; i < 16; ++i) {               // column 32 cb + 8 (i / 4) + 4 lh + i % 4
                const uint32_t here = static_cast<uint32_t>((i & 1 ? odd[rb] : even[rb]) >> (16 * cb + 4 * (i >> 2) + ((i & 3) >> 1))) & 1u;
                acc[cb][rb][i] += __uint_as_float(-here & 0x7FC00000u);   // NaN or nothing, without 128 conditions held at once
            }
    }
}

typedef int32_t int4v __attribute__((ext_vector_type(4)));
typedef int32_t int8v __attribute__((ext_vector_type(8)));

// Whether the handle's plan is of this call's numbers of tokens and sequences: not
// where a call is replayed from a graph after a plan of other sizes, whose items
// would lie outside its arrays.  Then nothing is done.
__device__ __forceinline__ bool planned(const DecodeArgs &a, int4v head) { return head[2] == a.n_tok && head[3] == a.n_seq; }

// This workgroup's item of a round (no item: n == 0) and its steps.
__device__ __forceinline__ DecodeItem take_item(const DecodeArgs &a, int round, bool &more, Shared &sh) {
    const int4v head = dev::ld_uniform(reinterpret_cast<const int4v *>(a.plan.head));
    const int8v v = dev::ld_uniform(reinterpret_cast<const int8v *>(a.plan.items + static_cast<int64_t>(round) * gridDim.x + blockIdx.x));
    DecodeItem it = __builtin_bit_cast(DecodeItem, v);
    more = it.seq & kItemMore;
    const bool prefix = it.seq & kItemPrefix;
    it.seq &= ~(kItemMore | kItemPrefix);
    if (__builtin_expect(!planned(a, head), 0)) {
        dev::flag_if(true, a.err, kErrSeq);
        it.n = 0;
        more = false;
    }
    sh.t0 = 2 * it.t0;
    sh.t1 = min(2 * it.t1, (it.len + kStepKeys - 1) / kStepKeys);
    sh.open = prefix ? INT32_MAX : it.len - it.n + (a.mask ? 0 : 1);
    return it;
}

template <bool BF, bool ONCE, bool Q8>
__global__ __launch_bounds__(kThreads, 2) void latent_decode_kernel(DecodeArgs a) {
    __shared__ __align__(1024) uint8_t s_kv[kKeyBytes<Q8> + kWeightBytes + (Q8 ? 8 * kRawBytes : 0)];
    __shared__ float s_red[2 * 2 * kTileRows], s_fac[kTileRows], s_sum[2 * kTileRows];
    __shared__ int s_raise[3], s_bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = dev::wave_id();
    const int l31 = lane & 31;
    const uint32_t kv_lds = dev::lds_address(s_kv);

    // The two kinds walk the items in loops of their own (and meet at the same
    // barriers): neither then holds registers for the other.
    bool more = true, bad_page = false;
    Shared sh{s_kv, s_kv + kKeyBytes<Q8>, s_kv + kKeyBytes<Q8> + kWeightBytes, s_red, s_fac, s_sum, s_raise, &s_bad, 0, 0, 0};
    if (wave < 4) {
        for (int round = 0; more; ++round) {
            const DecodeItem it = take_item(a, round, more, sh);
            if (it.n == 0) continue;
            const int rows = min(kTileRows, it.n * a.n_heads - it.row0);
            float m[2];
            for (int careful = 0; careful < 2; ++careful) {
                dev::lds_barrier();                      // the buffers of the item (or pass) before are free
                if (tid == 0) s_bad = s_raise[0] = s_raise[1] = s_raise[2] = 0;
                score_item<BF, Q8>(a, it, sh, rows, careful, m);
                dev::lds_barrier();
                if (!(s_bad && sh.t1 * kStepKeys > sh.open)) break;
            }
            if ((wave >> 1) == 0 && lane < 16)
#pragma unroll
                for (int rb = 0; rb < 2; ++rb) {
                    const int r = 32 * wave + lane + 16 * rb;
                    if (r >= rows) continue;
                    const float lr = s_sum[r] + s_sum[kTileRows + r];
                    if (it.slot >= 0) {
                        float *ml = a.part_ml + (static_cast<int64_t>(it.slot) * kTileRows + r) * 2;
                        ml[0] = m[rb];
                        ml[1] = lr;
                    } else if (a.lse) {
                        a.lse[static_cast<int64_t>(it.q0) * a.n_heads + it.row0 + r] =
                            lr == 0.0f ? -__builtin_inff() : (m[rb] + __builtin_amdgcn_logf(lr)) * kLn2;
                    }
                }
        }
    } else {
        const int w = wave - 4;
        for (int round = 0; more; ++round) {
            const DecodeItem it = take_item(a, round, more, sh);
            if (it.n == 0) continue;
            const int rows = min(kTileRows, it.n * a.n_heads - it.row0);
            f32x16 acc[4][2];                            // [32 columns][32 rows] blocks of O^T
            for (int careful = 0; careful < 2; ++careful) {
                dev::lds_barrier();
                sum_item<BF, ONCE, Q8>(a, it, sh, kv_lds, kv_lds + kKeyBytes<Q8> + kWeightBytes, rows, careful, bad_page, acc);
                if (careful) spoil_seen<BF, Q8>(a, it, sh, rows, acc);
                dev::lds_barrier();
                if (!(s_bad && sh.t1 * kStepKeys > sh.open)) break;
            }
            if (it.slot < 0) {
                const int64_t out_row = static_cast<int64_t>(it.q0) * a.n_heads + it.row0;
                const float l0 = s_sum[l31] + s_sum[kTileRows + l31], l1 = s_sum[32 + l31] + s_sum[kTileRows + 32 + l31];
                const float i0 = l0 == 0.0f ? 0.0f : 1.0f / l0, i1 = l1 == 0.0f ? 0.0f : 1.0f / l1;
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) {
                    uint8_t *o = a.out + ((out_row + l31) * kLatent + 128 * w + 32 * cb) * 2;
                    dev::store_tile16<BF>(acc[cb][0], i0, l31 < rows ? o : nullptr);
                    dev::store_tile16<BF>(acc[cb][1], i1, 32 + l31 < rows ? o + 32 * kLatent * 2 : nullptr);
                }
            } else {
                // Sixteen bytes per lane, a wave's 1 KB together (rows would
                // spread each store over 32 of them).  Of 32 rows or fewer the other half is
                // neither written nor read.
                f32x4 *part = reinterpret_cast<f32x4 *>(a.part + static_cast<int64_t>(it.slot) * kTileRows * kLatent) + w * 32 * 64 + lane;
#pragma unroll
                for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                    for (int rb = 0; rb < 2; ++rb) {
                        if (rb == 1 && rows <= 32) continue;
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            part[((cb * 2 + rb) * 4 + g) * 64] = f32x4{acc[cb][rb][4 * g], acc[cb][rb][4 * g + 1],
                                                                       acc[cb][rb][4 * g + 2], acc[cb][rb][4 * g + 3]};
                    }
            }
        }
    }
    dev::flag_if(bad_page, a.err, kErrPage);
}

// Joins the pieces of a row: with M = max m_i, o = sum 2^(m_i - M) O_i / sum
// 2^(m_i - M) l_i, summed in a fixed order.  A piece is 32 blocks of 4 KB as the
// summing waves held them: block (w 4 + cb) 2 + rb is rows 32 rb .. + 31 of
// columns 128 w + 32 cb .. + 31 as an accumulator, sixteen bytes of each lane at
// a time.  A wave joins one block of up to kWavePieces pieces, all of them in
// flight; of more the four waves of a workgroup take a quarter each and add up
// in LDS.
constexpr int kWavePieces = 8;
constexpr int kOutBlocks = kTileRows * kLatent / 1024;

template <bool BF>
__global__ __launch_bounds__(256) void join_kernel(DecodeArgs a) {
    __shared__ f32x4 s_o[3][4][64];
    __shared__ float s_l[3][64];
    const int4v head = dev::ld_uniform(reinterpret_cast<const int4v *>(a.plan.head));
    const int joins = planned(a, head) ? head[0] : 0, most = head[1];
    const bool apart = most <= kWavePieces;
    const int per = apart ? kOutBlocks / 4 : kOutBlocks;
    const int lane = threadIdx.x & 63, wave = dev::wave_id();
    for (int wg = blockIdx.x; wg < joins * per; wg += gridDim.x) {
        JoinUnit u = a.plan.joins[wg / per];
        const bool group = u.split & kJoinGroup;
        u.split &= ~kJoinGroup;
        const int block = apart ? 4 * (wg % per) + wave : wg % per;
        if (32 * (block & 1) >= u.rows) continue;         // (a workgroup's, where its waves meet)
        const int r = 32 * (block & 1) + (lane & 31);
        const bool live = r < u.rows;                     // partial rows past the unit's hold no statistics
        const float *ml = a.part_ml + (static_cast<int64_t>(u.slot0) * kTileRows + (live ? r : 0)) * 2;
        const f32x4 *part = reinterpret_cast<const f32x4 *>(a.part + static_cast<int64_t>(u.slot0) * kTileRows * kLatent) + block * 256 + lane;
        float top = -__builtin_inff();
#pragma unroll 8
        for (int i = 0; i < u.split; ++i) top = fmaxf(top, ml[i * kTileRows * 2]);
        // A group's rows: the pieces above are the prefix's, and each row has others, of its
        // own sequence, somewhere in that one's units.
        const float *oml = nullptr;
        const f32x4 *opart = nullptr;
        int own = 0, own_most = 0;
        if (group) {
            const int at = u.out_row + (live ? r : 0);
            const int4v rec = *reinterpret_cast<const int4v *>(a.plan.records + at / a.n_heads);
            const int in_seq = at - rec[2], orow = in_seq % kTileRows;
            const int64_t slot = rec[0] + in_seq / kTileRows * rec[1];
            own = rec[1];
            oml = a.part_ml + (slot * kTileRows + orow) * 2;
            opart = reinterpret_cast<const f32x4 *>(a.part + slot * kTileRows * kLatent) + ((block & ~1) | (orow >> 5)) * 256 + ((lane & 32) | (orow & 31));
            for (int i = 0; i < own; ++i) top = fmaxf(top, oml[i * kTileRows * 2]);
            own_most = own;
#pragma unroll
            for (int o = 32; o; o >>= 1) own_most = max(own_most, __shfl_xor(own_most, o, 64));
        }
        const float ms = top == -__builtin_inff() ? 0.0f : top;
        float l = 0.0f;
        f32x16 o;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = 0.0f;
        auto add = [&](const float *ml, const f32x4 *part, int i) {
            const float f = __builtin_amdgcn_exp2f(ml[i * kTileRows * 2] - ms);
            l = __builtin_fmaf(f, ml[i * kTileRows * 2 + 1], l);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 v = part[static_cast<int64_t>(i) * (kTileRows * kLatent / 4) + 64 * g];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[4 * g + j] = __builtin_fmaf(f, v[j], o[4 * g + j]);
            }
        };
        // The four waves of a workgroup take a quarter each of all pieces, the own ones first.
        const int all = own_most + u.split, p0 = apart ? 0 : all * wave / 4, p1 = apart ? all : all * (wave + 1) / 4;
        for (int i = p0; i < min(p1, own_most); ++i)
            if (i < own) add(oml, opart, i);
#pragma unroll 4
        for (int i = max(p0 - own_most, 0); i < p1 - own_most; ++i) add(ml, part, i);
        if (!apart) {
            __syncthreads();
            if (wave) {
#pragma unroll
                for (int g = 0; g < 4; ++g) s_o[wave - 1][g][lane] = f32x4{o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]};
                s_l[wave - 1][lane] = l;
            }
            __syncthreads();
            if (wave) continue;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                l += s_l[k][lane];
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[4 * g + j] += s_o[k][g][lane][j];
            }
        }
        const int64_t row = u.out_row + r;
        dev::store_tile16<BF>(o, l == 0.0f ? 0.0f : 1.0f / l, live ? a.out + (row * kLatent + 32 * (block >> 1)) * 2 : nullptr);
        if (a.lse && block < 2 && lane < 32 && live) a.lse[row] = l == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(l)) * kLn2;
    }
}

// The plan of a step, by one workgroup: each sequence's rows are cut into
// 64-row units and its key tiles into runs of at most `per`, the run length
// with the shortest estimated time.  One round over the CUs: the smallest run
// length that gives no more items than CUs, or a longer one, whose fewer pieces
// are joined the sooner: 16 pieces of one sequence, which a workgroup has in
// flight together, take most of a tile's time, and each piece a share of it (one
// token, 4096 keys: runs of two tiles 19.3 us, of four 20.3; 16384: two 36.3, four
// 28.7; 32768: two 50.9, eight 34.7; 16 tokens of 1000: two 27.7, four 24.4; 64 of
// 1000: four to eight 36.8, undivided 53.7).  Two to
// four rounds: the smallest that fits them; the sequences are then taken in the
// order of their runs' lengths and every other round is laid out backwards, so
// that the CUs' sums come close to their mean (16 ragged trees of 25 nodes:
// 45 + 45 tiles at most in the order of arrival, 71 so, at a mean of 64; 173 -> 154 us).
// Each item costs kItemCost tiles more, and joining the pieces a tile per
// kJoinItems.  With more units than four rounds hold, only units longer than a
// CU's fair share are cut.  A chain of latencies, once a step for all layers: 16 us
// for 64 sequences, 46 us for 1024 of four tokens.
constexpr int kPlanThreads = 1024;
constexpr int kItemCost = 3;    // tiles: the queries, the first tile's latency and the partial result
constexpr int kJoinItems = 64;  // pieces whose joining costs as much as a tile
constexpr int kMinRun = 2;
// (The costs are those of a 16-bit cache's tiles and of whole 64-row units; steps of an 8-bit
// cache and units of 32 rows or fewer take others, and pieces that are joined only because
// their prefix is shared are not counted: the plan does not know of them.)
constexpr float kTileTime = 1.4f, kPieceTime = 0.06f;   // of 16 pieces' joining
constexpr int kSortMost = 1024; // sequences that are put in order
static_assert(kPrefixEntries == kSortMost && kPrefixEntries == kPlanThreads, "an entry to a thread, all of them in LDS");
constexpr int kItemLanes = 16;  // lanes that write a sequence's items
constexpr int kLengthBits = 7, kLengths = 1 << kLengthBits;

__device__ __forceinline__ int cut(int tiles, int per) { return max(1, (tiles + per - 1) / per); }

// Groups of sequences that share a prefix (PREFIX).  The prefix is attended by an entry
// of its own behind the sequences' (at most kSortMost entries in all): the group's
// tokens, which are neighbours, are its rows, and its keys are the prefix's whole
// tiles, found through the first sequence's row of the block table.  No more than what
// every token of the group sees as context is shared, so that nothing of it is
// masked; the sequences begin behind it.  Both leave pieces for the join, which goes by
// the group's 64-row units and finds each row's own pieces by its token's record: by the
// sequences' units, of 16 rows each, it read the prefix's pieces four times over (64
// sequences behind 32000 tokens, 16 heads: 23 us, so 11).  That step: 89 us, 72 GF, 80 MB
// read; its plan 29 us, that of eight sequences behind 4096 tokens 15.
// Sharing saves products where the sequences' rows leave units partly empty, and costs an
// item, two pieces and their join for each unit; the plan does as it is told and does not weigh
// them.  One token and 500 of their own each, on the same pages, undivided and shared (us, the
// decode without its plan): 64 sequences of 16 heads behind 512 tokens 27 and 26, 4096 47
// and 31, 32000 213 and 88; of 64 heads, whose rows fill a unit by themselves, 31 and 30, 58 and
// 59, 289 and 268; 256 sequences behind 512 tokens 44 and 62 (16 heads), 52 and 83 (64).
struct Groups {
    const int32_t *start, *prefix;     // [n + 1] first sequences; [n] tokens
    int n;
};

template <bool PREFIX>
__global__ __launch_bounds__(kPlanThreads) void decode_plan_kernel(DecodePlan p, const int32_t *q_start, const int32_t *kv_len,
                                                                   int n_seq, int n_tok, int n_heads, int n_cu, int unit_cap,
                                                                   Groups groups, int32_t *err) {
    __shared__ int s_tmp[kPlanThreads / 64 + 1];
    __shared__ unsigned long long s_units, s_work;
    __shared__ float s_cost[kPlanThreads / 64];
    __shared__ int s_most, s_count[kPlanThreads / 64], s_order[kSortMost];
    __shared__ __align__(16) int s_key[kSortMost];
    // What the first sequences need, nearer than device memory: units, tiles,
    // first item and slot, and first token, tokens, length.
    __shared__ int4 s_seq[kSortMost], s_at[kSortMost];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, of_seq = n_seq;
    int4 *seq = reinterpret_cast<int4 *>(p.seq);         // units, tiles, first item, first slot
    if (tid == 0) {
        s_units = s_work = 0;
        s_most = 1;
    }
    __syncthreads();
    bool bad = false;
    unsigned long long my_units = 0, my_work = 0;
    int my_most = 1;
    // Of a sequence: its group (-1: none).  Of a group: first sequence and behind the
    // last, the least context of its tokens (later the tiles that it shares), how many
    // of its sequences have tokens, the first that does, and the most pieces of one.
    __shared__ int s_group[PREFIX ? kSortMost : 1], s_from[PREFIX ? kSortMost + 1 : 1], s_least[PREFIX ? kSortMost : 1], s_live[PREFIX ? kSortMost : 1], s_head[PREFIX ? kSortMost : 1];
    __shared__ int s_split[PREFIX ? kSortMost : 1];
    __shared__ int s_groups;
    const int q_seqs = n_seq;
    if constexpr (PREFIX) {
        if (tid == 0) s_groups = groups.n;
        if (tid <= groups.n) s_from[tid] = groups.start[tid];
        s_least[tid] = s_head[tid] = INT32_MAX;
        s_live[tid] = s_split[tid] = 0;
        __syncthreads();
        if (tid < groups.n && (s_from[tid] < 0 || s_from[tid + 1] < s_from[tid] || s_from[tid + 1] > n_seq)) {
            bad = true;
            s_groups = 0;                                // nothing is shared
        }
        __syncthreads();
        int g = -1;
        if (tid < n_seq && s_groups) {
            int lo = 0, hi = s_groups;                   // the last group that begins at or before the sequence
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (s_from[mid] <= tid) lo = mid + 1;
                else hi = mid;
            }
            if (lo > 0 && tid < s_from[lo]) g = lo - 1;
        }
        s_group[tid] = g;
        if (g >= 0) {
            const int q0 = q_start[tid], q1 = q_start[tid + 1], len = kv_len[tid];
            const bool ok = q0 >= 0 && q1 >= q0 && q1 <= n_tok && len >= 0 && len <= INT32_MAX - 2 * kTileKeys;
            if (!ok || q1 > q0) atomicMin(&s_least[g], ok ? len - (q1 - q0) : 0);
            if (ok && q1 > q0) {
                atomicAdd(&s_live[g], 1);
                atomicMin(&s_head[g], tid);
            }
        }
        __syncthreads();
        if (tid < groups.n) {
            const int g0 = s_from[tid];
            int tiles = 0, tokens = 0, q0 = 0;
            if (tid < s_groups && s_live[tid] > 1) {     // every sequence of the group is in order
                tiles = max(0, min(groups.prefix[tid], s_least[tid])) / kTileKeys;
                q0 = q_start[g0];
                tokens = tiles ? q_start[s_from[tid + 1]] - q0 : 0;
            }
            s_least[tid] = tiles;
            s_seq[n_seq + tid] = int4{static_cast<int>((static_cast<int64_t>(tokens) * n_heads + kTileRows - 1) / kTileRows), tiles, 0, 0};
            s_at[n_seq + tid] = int4{q0, tokens, tiles * kTileKeys, s_head[tid]};
        }
        __syncthreads();
    }
    for (int b = tid; b < n_seq; b += kPlanThreads) {
        const int q0 = q_start[b], q1 = q_start[b + 1], len = kv_len[b];
        const bool ok = q0 >= 0 && q1 >= q0 && q1 <= n_tok && len >= 0 && len <= INT32_MAX - 2 * kTileKeys;
        bad = bad || !ok;
        const int units = ok ? static_cast<int>((static_cast<int64_t>(q1 - q0) * n_heads + kTileRows - 1) / kTileRows) : 0;
        int tiles = ok ? (len + kTileKeys - 1) / kTileKeys : 0, behind = 0;
        if (PREFIX && s_group[b] >= 0 && units) behind = s_least[s_group[b]];
        tiles -= behind;
        if (b < kSortMost) {
            s_seq[b] = int4{units, tiles, 0, 0};
            s_at[b] = int4{q0, q1 - q0, len, behind};
        } else {
            seq[b] = int4{units, tiles, 0, 0};
        }
        my_units += units;
        my_work += static_cast<unsigned long long>(units) * tiles;
        if (units) my_most = max(my_most, tiles);
    }
    auto total = [&]() {
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            my_units += __shfl_xor(my_units, o, 64);
            my_work += __shfl_xor(my_work, o, 64);
            my_most = max(my_most, __shfl_xor(my_most, o, 64));
        }
        if (lane == 0) {
            atomicAdd(&s_units, my_units);
            atomicAdd(&s_work, my_work);
            atomicMax(&s_most, my_most);
        }
        __syncthreads();
    };
    if constexpr (PREFIX) {
        n_seq += groups.n;
        if (tid < groups.n) {
            const int4 s = s_seq[q_seqs + tid];
            my_units += s.x;
            my_work += static_cast<unsigned long long>(s.x) * s.y;
            if (s.x) my_most = max(my_most, s.y);
        }
    }
    total();
    if constexpr (PREFIX) {
        // A piece of every unit has to find room: else each sequence attends to all of its keys.
        if (s_units > static_cast<unsigned long long>(min(p.slot_cap, 4 * n_cu))) {
            n_seq = q_seqs;
            my_units = my_work = 0;
            my_most = 1;
            if (tid < n_seq) {
                s_seq[tid].y += s_at[tid].w;
                s_at[tid].w = 0;
                const int4 s = s_seq[tid];
                my_units = s.x;
                my_work = static_cast<unsigned long long>(s.x) * s.y;
                if (s.x) my_most = max(my_most, s.y);
            }
            __syncthreads();
            if (tid == 0) {
                s_units = s_work = 0;
                s_most = 1;
            }
            __syncthreads();
            total();
        }
    }
    const unsigned long long units = s_units;
    const int most = s_most;
    if (n_seq == q_seqs && units > static_cast<unsigned long long>(unit_cap)) {   // sequences that overlap: nothing is planned
        bad = true;
        n_seq = 0;
    }
    // Whether an entry's pieces are joined with others even if it is not cut.
    auto shares = [&](int b) { return PREFIX && (b >= q_seqs || s_at[b].w > 0); };
    // Items at a run length, one wave per candidate; 2^24 stands for any more.
    auto items_at = [&](int per) {
        unsigned long long n = 0;
        for (int b = lane; b < n_seq; b += 64) {
            const int4 s = b < kSortMost ? s_seq[b] : seq[b];
            n += static_cast<unsigned long long>(s.x) * cut(s.y, per);
        }
        const int sum = dev::running_sum(static_cast<int>(min(n, 1ull << 24)));
        return static_cast<unsigned long long>(__builtin_amdgcn_readlane(sum, 63));
    };
    int best = 0;
    long long best_cost = 0;
    int run1 = most, run2 = 0;                           // the smallest runs that fit one round and two
    for (int r = 1; r <= 4; ++r) {
        const unsigned long long room = static_cast<unsigned long long>(r) * n_cu;
        if (units > room) continue;
        int lo = min(kMinRun, most), hi = most;          // items_at(hi) == units <= room
        // work / run <= items <= work / run + units: what that leaves of the range,
        // with room for the roundings of the fp32 quotients.
        const float work = static_cast<float>(s_work);
        lo = static_cast<int>(fminf(fmaxf(0.9999f * work / static_cast<float>(room) - 1.0f, static_cast<float>(lo)), static_cast<float>(hi)));
        if (units < room) hi = max(lo, static_cast<int>(fminf(1.0001f * work / static_cast<float>(room - units) + 2.0f, static_cast<float>(hi))));
        while (lo < hi) {
            const int step = (hi - lo + 15) / 16;        // candidates lo + step * wave
            const int mine = min(lo + step * wave, hi);
            const bool fits = items_at(mine) <= room;
            if (lane == 0) s_count[wave] = fits;
            __syncthreads();
            // The first that fits: fits is monotone in the run length.
            const int w = __ffsll(__ballot(lane >= kPlanThreads / 64 || s_count[lane])) - 1;
            __syncthreads();
            const int top = w < 16 ? min(lo + step * w, hi) : hi;
            lo = w == 0 ? lo : min(lo + step * (w - 1) + 1, top);
            hi = top;
        }
        if (r == 1) run1 = hi;
        if (r == 2) run2 = hi;
        if (r == 1) {
            // The smallest that fits, or one up to 4.75 times as long whose fewer
            // pieces are joined the sooner.
            const int mine = static_cast<int>(min(hi + static_cast<long long>(hi) * wave / 4, static_cast<long long>(most)));
            const unsigned long long n = items_at(mine);
            const int depth = cut(most, mine);
            const float cost = kTileTime * static_cast<float>(mine) + (n == units ? 0.0f : static_cast<float>((depth + 15) / 16) + kPieceTime * static_cast<float>(n));
            if (lane == 0) s_cost[wave] = cost;
            __syncthreads();
            const float mycost = s_cost[lane & 15];
            float least = mycost;
#pragma unroll
            for (int o = 8; o; o >>= 1) least = fminf(least, __shfl_xor(least, o, 64));
            const int w = __ffsll(__ballot(mycost == least)) - 1;
            hi = static_cast<int>(min(hi + static_cast<long long>(hi) * w / 4, static_cast<long long>(most)));
        }
        const long long items = static_cast<long long>(items_at(hi));
        const long long each = r == 1 ? hi : max(static_cast<long long>(hi), static_cast<long long>(s_work / n_cu) + hi / 8);
        const long long cost = (each + static_cast<long long>(r) * kItemCost) * kJoinItems + (items > static_cast<long long>(units) ? items : 0);
        if (best == 0 || cost < best_cost) {
            best = hi;
            best_cost = cost;
        }
    }
    if constexpr (PREFIX) {
        // Prefixes give long runs beside the short ones of the sequences: between one round and
        // two lie runs of which the long ones have a CU each and the short ones share the
        // others.  Sixteen of them, a wave each, laid out on a histogram of the lengths.
        // (64 sequences of 20 to 2000 tokens behind 32000, 16 heads: the fullest CU 39
        // tiles, so 43 at a mean of 36, and 288 pieces, so 503.)
        if (run2 > 0 && run2 + 1 < run1) {
            __shared__ int s_hist[kPlanThreads / 64][kLengths];
            const int mine = run2 + 1 + static_cast<int>(static_cast<int64_t>(run1 - run2 - 1) * wave / (kPlanThreads / 64));
            const int scale = max(0, 32 - __clz(run1) - kLengthBits);
            int *hist = s_hist[wave];
            for (int i = lane; i < kLengths; i += 64) hist[i] = 0;
            __syncthreads();
            for (int b = lane; b < n_seq; b += 64) {
                const int4 v = s_seq[b];
                if (v.x == 0) continue;
                const int split = cut(v.y, mine), each = v.y / split, over = v.y - each * split;
                atomicAdd(hist + (each >> scale), v.x * (split - over));
                if (over) atomicAdd(hist + ((each + 1) >> scale), v.x * over);
            }
            __syncthreads();
            // How many are as long as each length: two of them a lane, from the longest down.
            static_assert(kLengths == 128, "two lengths a lane");
            const int at = kLengths - 1 - 2 * lane, longer = hist[at], here = longer + hist[at - 1], sum = dev::running_sum(here);
            hist[at] = sum - here + longer;
            hist[at - 1] = sum;
            __syncthreads();
            const int n = __builtin_amdgcn_readlane(sum, 63);
            auto load_of = [&](int i) {                  // of the i-th longest run
                if (i >= n) return 0.0f;
                int x = 0;
                for (int step = kLengths / 2; step; step >>= 1)
                    if (hist[x + step] > i) x += step;
                return static_cast<float>(((x + 1) << scale) - 1 + kItemCost);
            };
            float fullest = 0.0f;
            for (int k = lane; k < n_cu; k += 64) fullest = fmaxf(fullest, load_of(k) + load_of(2 * n_cu - 1 - k));
#pragma unroll
            for (int o = 32; o; o >>= 1) fullest = fmaxf(fullest, __shfl_xor(fullest, o, 64));
            if (lane == 0) s_cost[wave] = fullest * kJoinItems + static_cast<float>(n);
            __syncthreads();
            const float mycost = s_cost[lane & 15];
            float least = mycost;
#pragma unroll
            for (int o = 8; o; o >>= 1) least = fminf(least, __shfl_xor(least, o, 64));
            const int w = __ffsll(__ballot(mycost == least)) - 1;
            if (best == 0 || least < static_cast<float>(best_cost)) best = run2 + 1 + static_cast<int>(static_cast<int64_t>(run1 - run2 - 1) * w / (kPlanThreads / 64));
        }
    }
    if (best == 0) best = static_cast<int>((s_work + n_cu - 1) / n_cu);
    if (best < 1) best = 1;

    // With more than one round, the sequences by falling length of their runs.
    const bool sorted = n_seq <= kSortMost && items_at(best) > static_cast<unsigned long long>(n_cu);
    __syncthreads();
    if (sorted) {
        // By length, then by number, in one value (runs of 2^21 tiles or more tie).
        int mine = -1;
        if (tid < n_seq) {
            const int tiles = s_seq[tid].y, split = cut(tiles, best);
            mine = min((tiles + split - 1) / split, (1 << 21) - 1) * kSortMost + kSortMost - 1 - tid;
        }
        s_key[tid] = mine;
        __syncthreads();
        if (tid < n_seq) {
            int rank = 0;
            for (int b = 0; b < n_seq; b += 4) {
                const int4 k = *reinterpret_cast<const int4 *>(s_key + b);
                rank += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
            }
            s_order[rank] = tid;
        }
    }
    int n_items = 0, n_slots = 0, n_joins = 0;
    if (tid == 0) s_most = 1;
    __syncthreads();
    for (int b0 = 0; b0 < n_seq; b0 += kPlanThreads) {
        const int b = b0 + tid >= n_seq ? n_seq : sorted ? s_order[b0 + tid] : b0 + tid;
        int4 s = b >= n_seq ? int4{0, 0, 0, 0} : b < kSortMost ? s_seq[b] : seq[b];
        const int split = cut(s.y, best), count = s.x * split;
        const bool parts = b < n_seq && (split > 1 || shares(b));
        // Rows of a group are joined in its units, those of other sequences in their own.
        const int units_joined = parts && (!PREFIX || b >= q_seqs || s_at[b].w == 0) ? s.x : 0;
        int total;
        const int at = n_items + dev::block_exclusive_scan<kPlanThreads>(count, s_tmp, &total);
        n_items += total;
        const int slot = n_slots + dev::block_exclusive_scan<kPlanThreads>(parts ? count : 0, s_tmp, &total);
        n_slots += total;
        const int join = n_joins + dev::block_exclusive_scan<kPlanThreads>(units_joined, s_tmp, &total);
        n_joins += total;
        if (b < n_seq) {
            s.z = at;
            s.w = parts ? slot : -1;
            if (b < kSortMost) s_seq[b] = s;
            else seq[b] = s;
        }
        if (PREFIX && parts && b < q_seqs && s_at[b].w > 0 && s.x) atomicMax(&s_split[s_group[b]], split);
        if constexpr (PREFIX) __syncthreads();           // the groups' longest divisions
        if (units_joined) {
            const bool group = PREFIX && b >= q_seqs;
            JoinUnit u{};
            atomicMax(&s_most, split + (group ? s_split[b - q_seqs] : 0));
            if (slot + count <= p.slot_cap && join + s.x <= p.join_cap) {
                const int q0 = b < kSortMost ? s_at[b].x : q_start[b], rows = (b < kSortMost ? s_at[b].y : q_start[b + 1] - q0) * n_heads;
                u.split = split | (group ? kJoinGroup : 0);
                for (int i = 0; i < s.x; ++i) {
                    u.out_row = q0 * n_heads + i * kTileRows;
                    u.rows = min(kTileRows, rows - i * kTileRows);
                    u.slot0 = slot + i * split;
                    p.joins[join + i] = u;
                }
            }
        }
    }
    // Round r, place x: workgroup x runs on XCD x % 8, and neighbouring items
    // share keys, so a round's items lie in eight contiguous runs, one per XCD.
    // Of more rounds than one, every other is laid out backwards.
    const int rounds = max(1, (n_items + n_cu - 1) / n_cu);
    const bool fits = rounds * n_cu <= p.item_cap && n_slots <= p.slot_cap && n_joins <= p.join_cap;
    const int run = rounds > 1 ? n_cu / 8 : (n_items + 7) / 8;
    auto place = [&](int i) {
        const int r = i / n_cu, at = (r & 1) ? n_cu - 1 - (i - r * n_cu) : i - r * n_cu;
        return r * n_cu + (at % run) * 8 + at / run;
    };
    __syncthreads();
    for (int i = tid; i < (fits ? rounds : 1) * n_cu; i += kPlanThreads) {
        const int r = i / n_cu, x = i - r * n_cu, here = fits ? min(n_cu, n_items - r * n_cu) : 0;
        const int pos = (x & 7) * run + (x >> 3), at = (r & 1) ? n_cu - 1 - pos : pos;
        if ((x >> 3) >= run || at >= here) {
            DecodeItem none{};
            none.seq = r + 1 < rounds && fits ? kItemMore : 0;
            p.items[i] = none;
        }
    }
    if (fits)
        for (int b = tid / kItemLanes; b < n_seq; b += kPlanThreads / kItemLanes) {
            int4 s, at;
            if (b < kSortMost) {
                s = s_seq[b];
                at = s_at[b];
            } else {
                s = seq[b];
                at = int4{q_start[b], q_start[b + 1] - q_start[b], kv_len[b], 0};
            }
            const bool prefix = PREFIX && b >= q_seqs;
            const int behind = PREFIX && !prefix ? at.w : 0, seq_bits = prefix ? at.w | kItemPrefix : b;
            const int split = cut(s.y, best), each = s.y / split, over = s.y - each * split;
            if (PREFIX && !prefix && behind)              // where the join finds the pieces of a token's rows
                for (int i = tid % kItemLanes; i < at.y; i += kItemLanes) p.records[at.x + i] = int4v{s.w, split, at.x * n_heads, 0};
            // Neighbouring items: the units of one run of keys.
            for (int i = tid % kItemLanes; i < s.x * split; i += kItemLanes) {
                const int c = i / s.x, u = i - c * s.x;
                DecodeItem it;
                it.q0 = at.x;
                it.n = at.y;
                it.len = at.z;
                it.seq = seq_bits | ((s.z + i) / n_cu + 1 < rounds ? kItemMore : 0);
                it.row0 = u * kTileRows;
                it.t0 = behind + c * each + min(c, over);
                it.t1 = it.t0 + each + (c < over);
                it.slot = s.w < 0 ? -1 : s.w + u * split + c;
                p.items[place(s.z + i)] = it;
            }
        }
    if (tid == 0) {
        p.head[0] = fits ? n_joins : 0;
        p.head[1] = s_most;
        p.head[2] = n_tok;
        p.head[3] = of_seq;
    }
    dev::flag_if(bad || !fits, err, kErrSeq);
}

}  // namespace

hipError_t launch_decode_plan(const DecodePlan &p, const int32_t *q_start, const int32_t *kv_len, int n_seq, int n_tok,
                              int n_heads, int n_cu, const int32_t *group_start, const int32_t *prefix_len, int n_groups, int32_t *err,
                              hipStream_t s) {
    const int unit_cap = static_cast<int>(std::min<int64_t>(INT32_MAX, static_cast<int64_t>(n_tok) * n_heads / kTileRows + n_seq));
    const Groups groups{group_start, prefix_len, n_groups};
    launch(n_groups ? decode_plan_kernel<true> : decode_plan_kernel<false>, 1u, kPlanThreads, 0, s, p, q_start, kv_len, n_seq, n_tok, n_heads, n_cu, unit_cap,
           groups, err);
    return hipGetLastError();
}

template <bool Q8>
static void launch_decode_kernel(const DecodeArgs &a, bool bf16, bool once, int n_cu, hipStream_t s) {
    launch(once ? (bf16 ? latent_decode_kernel<true, true, Q8> : latent_decode_kernel<false, true, Q8>)
                : (bf16 ? latent_decode_kernel<true, false, Q8> : latent_decode_kernel<false, false, Q8>),
           static_cast<unsigned>(n_cu), kThreads, 0, s, a);
}

hipError_t launch_latent_decode(const DecodeArgs &a, bool bf16, bool cache8, bool prefixes, int n_cu, hipStream_t s) {
    // Where a sequence's rows fill one item (on the average: the sequences' own
    // counts are the device's), its keys are read once and not kept in the
    // caches: 64 sequences up to 12k tokens 88 -> 81 us.  Items that share keys
    // lose by it (trees of 25 nodes 173 -> 178 us), and by a test at each
    // copy instead of two kernels (191 us).
    const bool once = !prefixes && static_cast<int64_t>(a.n_tok) * a.n_heads <= static_cast<int64_t>(a.n_seq) * kTileRows;
    if (cache8) launch_decode_kernel<true>(a, bf16, once, n_cu, s);
    else launch_decode_kernel<false>(a, bf16, once, n_cu, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(a.join_most) * kOutBlocks, 8 * n_cu));
    launch(bf16 ? join_kernel<true> : join_kernel<false>, blocks, 256u, 0, s, a);
    return hipGetLastError();
}

}  // namespace coli
