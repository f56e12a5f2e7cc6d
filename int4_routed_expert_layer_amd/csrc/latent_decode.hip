// latent_decode.hip -- absorbed latent attention of single, chained or
// tree-drafted tokens over the paged latent cache.
//
// Every head of a token attends to the same 576 cached values per key (512
// latent ones that are key and value, 64 rotary ones that are key only):
//   s_j = scale (q_lat . c_j + q_pe . r_j),  o = sum_j softmax(s)_j c_j,
// so the (token, head) pairs of a sequence are rows of one product and a key
// is read once for 64 of them.  One workgroup (four waves, one per SIMD, a CU
// to itself) takes 64 rows and a run of 64-key tiles, with the running
// maximum and sum of the softmax:
//   - the tile (72 KB) is copied straight into LDS, double buffered; the copy
//     of tile t + 1 is in flight while tile t is used;
//   - S^T = K Q^T: wave (wm, wk) computes 32 keys x 32 rows with its rows'
//     queries held in 144 registers, so lane L of a wave owns row L % 32;
//   - the maxima of the two key halves and the 16-bit probabilities are
//     exchanged through LDS;
//   - O^T += V^T P^T: each wave computes all 64 rows of 128 latent columns
//     (128 accumulator registers), reading V^T with transposed LDS reads.
// Splitting the keys of the first product and the columns of the second means
// that each wave reads half of K and a quarter of V from LDS; with rows alone
// split every wave would read all of both.
//
// A sequence's keys are cut into pieces so that every CU has one (the plan);
// pieces leave unnormalised sums, maxima and fp32 partial outputs, which
// join_kernel combines.
#include "dev_attn.h"

namespace coli {
namespace {

using dev::f32x16;
using dev::f32x4;
using dev::u32x2;
using dev::u32x4;

constexpr int kBlocks = kCacheRow / 64;                  // 64-column blocks of a cached row: 8 latent, 1 rotary
constexpr int kLatentBlocks = kLatent / 64;
constexpr int kBlockBytes = kTileKeys * 128;
constexpr int kTileBytes = kBlocks * kBlockBytes;        // 72 KB
constexpr int kSteps = kCacheRow / 16;                   // K steps of the first product
// The running maximum of a row moves only when a tile exceeds it by more than
// 2^kSlack: the accumulator is then rarely rescaled, and probabilities stay
// below 2^kSlack, far inside the range of both 16-bit types and of the sums.
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

// Which 64 keys of a tile a row sees, as bits.  Rows of a chain see keys up to
// their own position; rows of a tree see the context and the nodes of their
// ancestor bits.
__device__ __forceinline__ uint64_t below(int c) { return c >= 64 ? ~0ull : c <= 0 ? 0ull : (1ull << c) - 1; }
__device__ __forceinline__ uint64_t seen_keys(const DecodeArgs &a, const DecodeItem &it, int node, int t) {
    const int ctx = it.len - it.n, key0 = t * kTileKeys;
    if (!a.mask) return below(ctx + node + 1 - key0);
    const uint64_t *m = a.mask + static_cast<int64_t>(it.q0 + node) * a.mask_words;
    const int d = key0 - ctx;                            // node index of the tile's first key
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

template <bool BF>
__global__ __launch_bounds__(256, 1) void latent_decode_kernel(DecodeArgs a) {
    __shared__ __align__(1024) uint8_t s_kv[2 * kTileBytes];
    __shared__ __align__(1024) uint8_t s_p[kTileRows * 128];
    __shared__ float s_red[2][kTileRows];
    __shared__ float s_fac[kTileRows];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = dev::wave_id();
    const int wm = wave & 1, wk = wave >> 1;
    const int l31 = lane & 31, lh = lane >> 5;
    const uint32_t kv_lds = dev::lds_address(s_kv);
    const float c = a.scale * kLog2e;

    const int n_items = dev::ld_uniform(a.plan.head);
    const int grid = static_cast<int>(gridDim.x);
    for (int first = 0; first < n_items; first += grid) {
        // Neighbouring items share keys: eight contiguous runs, one per XCD.
        const int here = min(grid, n_items - first), run = (here + 7) / 8;
        const int bx = static_cast<int>(blockIdx.x) & 7, by = static_cast<int>(blockIdx.x) >> 3;
        if (by >= run || bx * run + by >= here) continue;
        typedef int32_t int8v __attribute__((ext_vector_type(8)));
        const DecodeItem it = __builtin_bit_cast(
            DecodeItem, dev::ld_uniform(reinterpret_cast<const int8v *>(a.plan.items + first + bx * run + by)));
        const int rows = min(kTileRows, it.n * a.n_heads - it.row0);
        const int row = 32 * wm + l31;                   // the row this lane scores
        const int rr = it.row0 + min(row, rows - 1);
        const int node = rr / a.n_heads, head = rr - node * a.n_heads;

        // Copies: per tile this lane fetches one 16-byte unit of each block of
        // two keys; their page numbers are read one tile ahead.
        const int cr = 16 * wave + (lane >> 3);
        const int32_t *table = a.cache.table + it.seq * a.cache.table_stride;
        bool bad_page = false;
        auto page_of = [&](int t, int j) {
            const int pos = min(t * kTileKeys + cr + 8 * j, it.len - 1), at = pos >> a.cache.page_shift;
            int pg = at < a.cache.table_cols ? table[at] : -1;
            if (pg < 0 || pg >= a.cache.n_pages) {
                bad_page = true;
                pg = 0;
            }
            return pg;
        };
        auto copy_tile = [&](int t, int buf, const int (&pg)[2]) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int pos = min(t * kTileKeys + cr + 8 * j, it.len - 1);
                const int in = pos & ((1 << a.cache.page_shift) - 1);
                const uint8_t *src = a.cache.base + (pg[j] * a.cache.page_stride + static_cast<int64_t>(in) * kCacheRow) * 2 +
                                     (((lane & 7) ^ dev::tile_swz(8 * j + (lane >> 3))) << 4);
                const uint32_t dst = kv_lds + buf * kTileBytes + (2 * wave + j) * 1024;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) dev::copy16_to_lds(src + b * 128, dst + b * kBlockBytes);
            }
        };

        u32x4 q[kSteps];
        {
            const int64_t tok = it.q0 + node;
            const uint8_t *ql = a.q_lat + (tok * a.ql_tok + head * a.ql_head) * 2 + 16 * lh;
            const uint8_t *qp = a.q_pe + (tok * a.qp_tok + head * a.qp_head) * 2 + 16 * lh;
#pragma unroll
            for (int k = 0; k < kLatent / 16; ++k) q[k] = dev::gload<u32x4>(ql + 32 * k);
#pragma unroll
            for (int k = kLatent / 16; k < kSteps; ++k) q[k] = dev::gload<u32x4>(qp + 32 * (k - kLatent / 16));
        }

        const int ctx = it.len - it.n;
        const int open = ctx + (a.mask ? 0 : 1);         // keys below are seen by every row
        f32x16 acc[4][2];                                // [32 columns][32 rows] blocks of O^T
        float m, l;
        for (int careful = 0; careful < 2; ++careful) {
#pragma unroll
            for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                for (int rb = 0; rb < 2; ++rb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[cb][rb][i] = 0.0f;
            m = -__builtin_inff();
            l = 0.0f;
            dev::lds_barrier();                          // the buffers of the item (or pass) before are free
            if (tid == 0) s_bad = 0;
            int pg[2] = {0, 0};
            if (it.t0 < it.t1) {
                const int now[2] = {page_of(it.t0, 0), page_of(it.t0, 1)};
                copy_tile(it.t0, 0, now);
                if (it.t0 + 1 < it.t1) {
                    pg[0] = page_of(it.t0 + 1, 0);
                    pg[1] = page_of(it.t0 + 1, 1);
                }
            }
            for (int t = it.t0; t < it.t1; ++t) {
                const int buf = (t - it.t0) & 1;
                uint8_t *kv = s_kv + buf * kTileBytes;
                dev::copy_barrier();
                if (t + 1 < it.t1) {
                    copy_tile(t + 1, buf ^ 1, pg);
                    if (t + 2 < it.t1) {
                        pg[0] = page_of(t + 2, 0);
                        pg[1] = page_of(t + 2, 1);
                    }
                }
                // S^T of 32 keys (wk) x 32 rows (wm), in two chains.
                f32x16 s0, s1;
#pragma unroll
                for (int i = 0; i < 16; ++i) s0[i] = s1[i] = 0.0f;
                const uint8_t *kr = kv + 32 * wk * 128;
#pragma unroll
                for (int k = 0; k < kSteps; k += 2) {
                    const uint8_t *blk = kr + (k >> 2) * kBlockBytes;
                    const u32x4 k0 = *reinterpret_cast<const u32x4 *>(blk + dev::tile_unit(l31, 2 * (k & 3) + lh));
                    const u32x4 k1 = *reinterpret_cast<const u32x4 *>(blk + dev::tile_unit(l31, 2 * ((k + 1) & 3) + lh));
                    s0 = dev::mma<BF>(k0, q[k], s0);
                    s1 = dev::mma<BF>(k1, q[k + 1], s1);
                }
                const bool masked = (t + 1) * kTileKeys > open;
#pragma unroll
                for (int i = 0; i < 16; ++i) s0[i] += s1[i];
                if (masked) {
                    const uint64_t seen = seen_keys(a, it, node, t) >> (32 * wk + 4 * lh);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!((seen >> (8 * (i >> 2) + (i & 3))) & 1)) s0[i] = -__builtin_inff();
                }
                float mx = s0[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s0[i]);
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                if (lh == 0) s_red[wk][row] = mx;
                dev::lds_barrier();
                const float tm = fmaxf(mx, s_red[wk ^ 1][row]) * c;
                const float m1 = tm > m + kSlack ? tm : m;
                const float fac = m1 == m ? 1.0f : __builtin_amdgcn_exp2f(m - m1);
                m = m1;
                const float ms = m1 == -__builtin_inff() ? 0.0f : m1;
                float sum = 0.0f;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s0[4 * g + j], c, -ms));
                        sum += p[j];
                    }
                    *reinterpret_cast<u32x2 *>(s_p + dev::tile_unit(row, 4 * wk + g) + 8 * lh) =
                        u32x2{dev::pack2<BF>(p[0], p[1]), dev::pack2<BF>(p[2], p[3])};
                }
                l = l * fac + sum;
                if (wk == 0 && lh == 0) s_fac[row] = fac;
                if (careful && masked) {
                    // Rows a tile hides hold what other branches left there:
                    // their weight is zero, and zero times inf or NaN must not
                    // reach this row.  (A row that sees such a key already has
                    // a NaN score.)
                    u32x4 *v = reinterpret_cast<u32x4 *>(kv);
                    for (int i = tid; i < kLatentBlocks * kBlockBytes / 16; i += 256) {
                        u32x4 w = v[i];
#pragma unroll
                        for (int d = 0; d < 4; ++d) w[d] &= ~dev::nonfinite_halves<BF>(w[d]);
                        v[i] = w;
                    }
                }
                dev::lds_barrier();
                const float f0 = s_fac[l31], f1 = s_fac[32 + l31];
                if (__any(f0 != 1.0f || f1 != 1.0f)) {
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            acc[cb][0][i] *= f0;
                            acc[cb][1][i] *= f1;
                        }
                }
                // O^T: columns 128 wave .. + 127, 16 keys per step.
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const u32x4 p0 = *reinterpret_cast<const u32x4 *>(s_p + dev::tile_unit(l31, 2 * k + lh));
                    const u32x4 p1 = *reinterpret_cast<const u32x4 *>(s_p + dev::tile_unit(32 + l31, 2 * k + lh));
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) {
                        const uint8_t *blk = kv + (2 * wave + (cb >> 1)) * kBlockBytes + 16 * k * 128;
                        const int unit = 4 * (cb & 1) + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
                        const int kr0 = 8 * lh + ((lane >> 2) & 3);
                        const u32x2 a0 = dev::read_tr(blk + dev::tile_unit(kr0, unit) + 8 * (lane & 1));
                        const u32x2 a1 = dev::read_tr(blk + dev::tile_unit(kr0 + 4, unit) + 8 * (lane & 1));
                        const u32x4 v = {a0[0], a0[1], a1[0], a1[1]};
                        acc[cb][0] = dev::mma<BF>(v, p0, acc[cb][0]);
                        acc[cb][1] = dev::mma<BF>(v, p1, acc[cb][1]);
                    }
                }
            }
            // The row sums of both key halves; whether anything is not finite.
            l += __shfl_xor(l, 32, 64);
            dev::lds_barrier();
            if (lh == 0) s_red[wk][row] = l;
            float z = 0.0f;
#pragma unroll
            for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                for (int rb = 0; rb < 2; ++rb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) z = __builtin_fmaf(acc[cb][rb][i], 0.0f, z);
            if (__any(z != 0.0f)) s_bad = 1;
            dev::lds_barrier();
            if (!(s_bad && it.t1 * kTileKeys > open)) break;
        }

        const float l0 = s_red[0][l31] + s_red[1][l31], l1 = s_red[0][32 + l31] + s_red[1][32 + l31];
        const int64_t out_row = static_cast<int64_t>(it.q0) * a.n_heads + it.row0;
        if (it.slot < 0) {
            const float i0 = l0 == 0.0f ? 0.0f : 1.0f / l0, i1 = l1 == 0.0f ? 0.0f : 1.0f / l1;
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
                const int col = 128 * wave + 32 * cb;
                uint8_t *o = a.out + ((out_row + l31) * kLatent + col) * 2;
                dev::store_tile16<BF>(acc[cb][0], i0, l31 < rows ? o : nullptr);
                dev::store_tile16<BF>(acc[cb][1], i1, 32 + l31 < rows ? o + 32 * kLatent * 2 : nullptr);
            }
            if (a.lse && wk == 0 && lh == 0 && row < rows) {
                const float lr = wm ? l1 : l0;
                a.lse[out_row + row] = lr == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(lr)) * kLn2;
            }
        } else {
            float *part = a.part + static_cast<int64_t>(it.slot) * kTileRows * kLatent;
#pragma unroll
            for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                for (int rb = 0; rb < 2; ++rb)
                    if (32 * rb + l31 < rows) {
                        float *o = part + (32 * rb + l31) * kLatent + 128 * wave + 32 * cb + 4 * lh;
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            *reinterpret_cast<f32x4 *>(o + 8 * g) = f32x4{acc[cb][rb][4 * g], acc[cb][rb][4 * g + 1],
                                                                          acc[cb][rb][4 * g + 2], acc[cb][rb][4 * g + 3]};
                    }
            if (wk == 0 && lh == 0 && row < rows) {
                float *ml = a.part_ml + (static_cast<int64_t>(it.slot) * kTileRows + row) * 2;
                ml[0] = m;
                ml[1] = wm ? l1 : l0;
            }
        }
        dev::flag_if(bad_page, a.err, kErrPage);
    }
}

// Joins the pieces of a row: with M = max m_i, o = sum 2^(m_i - M) O_i / sum
// 2^(m_i - M) l_i.  Two rows per 256-thread workgroup, four columns per
// thread; the pieces of one row are read in a fixed order.
template <bool BF>
__global__ __launch_bounds__(256) void join_kernel(DecodeArgs a) {
    const int n = dev::ld_uniform(a.plan.head + 1) * (kTileRows / 2);
    const int half = threadIdx.x >> 7, col = 4 * (threadIdx.x & 127);
    for (int w = blockIdx.x; w < n; w += gridDim.x) {
        const JoinUnit u = a.plan.joins[w / (kTileRows / 2)];
        const int r = 2 * (w % (kTileRows / 2)) + half;
        if (r >= u.rows) continue;
        const float *ml = a.part_ml + (static_cast<int64_t>(u.slot0) * kTileRows + r) * 2;
        const float *part = a.part + (static_cast<int64_t>(u.slot0) * kTileRows + r) * kLatent + col;
        float top = -__builtin_inff();
        for (int i = 0; i < u.split; ++i) top = fmaxf(top, ml[i * kTileRows * 2]);
        const float ms = top == -__builtin_inff() ? 0.0f : top;
        float l = 0.0f;
        f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int i = 0; i < u.split; ++i) {
            const float f = __builtin_amdgcn_exp2f(ml[i * kTileRows * 2] - ms);
            const f32x4 v = *reinterpret_cast<const f32x4 *>(part + static_cast<int64_t>(i) * kTileRows * kLatent);
            l = __builtin_fmaf(f, ml[i * kTileRows * 2 + 1], l);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = __builtin_fmaf(f, v[j], o[j]);
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t row = u.out_row + r;
        *reinterpret_cast<u32x2 *>(a.out + (row * kLatent + col) * 2) =
            u32x2{dev::pack2<BF>(o[0] * inv, o[1] * inv), dev::pack2<BF>(o[2] * inv, o[3] * inv)};
        if (a.lse && col == 0) a.lse[row] = l == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(l)) * kLn2;
    }
}

// The plan of a step, by one workgroup: each sequence's rows are cut into
// 64-row units and its key tiles into runs of at most `per`, the run length
// with the shortest estimated time: for one to four rounds over the CUs the
// smallest run length that fits that many rounds, at (per + kItemCost) per
// round.  With more units than four rounds hold, only units longer than a
// CU's fair share are cut.
constexpr int kPlanThreads = 1024;
constexpr int kItemCost = 3;    // tiles: the queries, the first tile's latency and the partial result
constexpr int kMinRun = 2;

__device__ __forceinline__ int cut(int tiles, int per) { return max(1, (tiles + per - 1) / per); }

__global__ __launch_bounds__(kPlanThreads) void decode_plan_kernel(DecodePlan p, const int32_t *q_start, const int32_t *kv_len,
                                                                   int n_seq, int n_tok, int n_heads, int n_cu, int unit_cap,
                                                                   int32_t *err) {
    __shared__ int s_tmp[kPlanThreads / 64 + 1];
    __shared__ unsigned long long s_units, s_work;
    __shared__ int s_most, s_count[kPlanThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int4 *seq = reinterpret_cast<int4 *>(p.seq);         // units, tiles, first item, first slot
    if (tid == 0) {
        s_units = s_work = 0;
        s_most = 1;
    }
    __syncthreads();
    bool bad = false;
    for (int b = tid; b < n_seq; b += kPlanThreads) {
        const int q0 = q_start[b], q1 = q_start[b + 1], len = kv_len[b];
        const bool ok = q0 >= 0 && q1 >= q0 && q1 <= n_tok && len >= 0 && len <= INT32_MAX - 2 * kTileKeys;
        bad = bad || !ok;
        const int units = ok ? static_cast<int>((static_cast<int64_t>(q1 - q0) * n_heads + kTileRows - 1) / kTileRows) : 0;
        const int tiles = ok ? (len + kTileKeys - 1) / kTileKeys : 0;
        seq[b] = int4{units, tiles, 0, 0};
        atomicAdd(&s_units, static_cast<unsigned long long>(units));
        atomicAdd(&s_work, static_cast<unsigned long long>(units) * tiles);
        if (units) atomicMax(&s_most, tiles);
    }
    __syncthreads();
    const unsigned long long units = s_units;
    const int most = s_most;
    if (units > static_cast<unsigned long long>(unit_cap)) {   // sequences that overlap: nothing is planned
        bad = true;
        n_seq = 0;
    }
    // Items at a run length, one wave per candidate.
    auto items_at = [&](int per) {
        unsigned long long n = 0;
        for (int b = lane; b < n_seq; b += 64) n += static_cast<unsigned long long>(seq[b].x) * cut(seq[b].y, per);
#pragma unroll
        for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o, 64);
        return n;
    };
    int best = 0;
    long long best_cost = 0;
    for (int r = 1; r <= 4; ++r) {
        const unsigned long long room = static_cast<unsigned long long>(r) * n_cu;
        if (units > room) continue;
        int lo = min(kMinRun, most), hi = most;          // items_at(hi) == units <= room
        while (lo < hi) {
            const int step = (hi - lo + 15) / 16;        // candidates lo + step * wave
            const int mine = min(lo + step * wave, hi);
            const bool fits = items_at(mine) <= room;
            if (lane == 0) s_count[wave] = fits;
            __syncthreads();
            int w = 0;
            while (w < 16 && !s_count[w]) ++w;           // fits is monotone in the run length
            __syncthreads();
            const int top = w < 16 ? min(lo + step * w, hi) : hi;
            lo = w == 0 ? lo : min(lo + step * (w - 1) + 1, top);
            hi = top;
        }
        const long long cost = static_cast<long long>(r) * (hi + kItemCost);
        if (best == 0 || cost < best_cost) {
            best = hi;
            best_cost = cost;
        }
    }
    if (best == 0) best = static_cast<int>((s_work + n_cu - 1) / n_cu);
    if (best < 1) best = 1;

    int n_items = 0, n_slots = 0, n_joins = 0;
    for (int b0 = 0; b0 < n_seq; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int4 s = b < n_seq ? seq[b] : int4{0, 0, 0, 0};
        const int split = cut(s.y, best), count = s.x * split;
        int total;
        const int at = n_items + dev::block_exclusive_scan<kPlanThreads>(count, s_tmp, &total);
        n_items += total;
        const int slot = n_slots + dev::block_exclusive_scan<kPlanThreads>(split > 1 ? count : 0, s_tmp, &total);
        n_slots += total;
        const int join = n_joins + dev::block_exclusive_scan<kPlanThreads>(split > 1 ? s.x : 0, s_tmp, &total);
        n_joins += total;
        if (b < n_seq) {
            s.z = at;
            s.w = split > 1 ? slot : -1;
            seq[b] = s;
            if (split > 1 && slot + count <= p.slot_cap) {
                const int q0 = q_start[b], rows = (q_start[b + 1] - q0) * n_heads;
                for (int i = 0; i < s.x; ++i)
                    p.joins[join + i] = JoinUnit{q0 * n_heads + i * kTileRows, min(kTileRows, rows - i * kTileRows), slot + i * split, split};
            }
        }
    }
    const bool fits = n_items <= p.item_cap && n_slots <= p.slot_cap;
    __syncthreads();
    if (fits)
        for (int b = wave; b < n_seq; b += kPlanThreads / 64) {
            const int4 s = seq[b];
            const int split = cut(s.y, best), q0 = q_start[b], n = q_start[b + 1] - q0, len = kv_len[b];
            // Neighbouring items: the units of one run of keys.
            for (int i = lane; i < s.x * split; i += 64) {
                const int c = i / s.x, u = i - c * s.x;
                DecodeItem it;
                it.q0 = q0;
                it.n = n;
                it.len = len;
                it.seq = b;
                it.row0 = u * kTileRows;
                it.t0 = static_cast<int>(static_cast<int64_t>(s.y) * c / split);
                it.t1 = static_cast<int>(static_cast<int64_t>(s.y) * (c + 1) / split);
                it.slot = s.w < 0 ? -1 : s.w + u * split + c;
                p.items[s.z + i] = it;
            }
        }
    if (tid == 0) {
        p.head[0] = fits ? n_items : 0;
        p.head[1] = fits ? n_joins : 0;
    }
    dev::flag_if(bad || !fits, err, kErrSeq);
}

}  // namespace

hipError_t launch_decode_plan(const DecodePlan &p, const int32_t *q_start, const int32_t *kv_len, int n_seq, int n_tok,
                              int n_heads, int n_cu, int32_t *err, hipStream_t s) {
    const int unit_cap = static_cast<int>(std::min<int64_t>(INT32_MAX, static_cast<int64_t>(n_tok) * n_heads / kTileRows + n_seq));
    launch(decode_plan_kernel, 1u, kPlanThreads, 0, s, p, q_start, kv_len, n_seq, n_tok, n_heads, n_cu, unit_cap, err);
    return hipGetLastError();
}

hipError_t launch_latent_decode(const DecodeArgs &a, bool bf16, int n_cu, hipStream_t s) {
    launch(bf16 ? latent_decode_kernel<true> : latent_decode_kernel<false>, static_cast<unsigned>(n_cu), 256u, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    launch(bf16 ? join_kernel<true> : join_kernel<false>, static_cast<unsigned>(2 * n_cu), 256u, 0, s, a);
    return hipGetLastError();
}

}  // namespace coli
