// latent_prompt.hip -- expanded latent attention of whole prompts: per-head
// keys and values from the up-projection, one rotary key shared by the heads.
//
//   s_j = scale (q_nope . k_j + q_pe . r_j),  o = sum_j softmax(s)_j v_j,
// causal with the queries as the last tokens of their sequence.  k_j and v_j
// are read where the up-projection left them ([token][head][nope + v]) and the
// rotary part from its own rows, so no key is ever assembled in memory.
//
// The narrow head: a wave takes 32 query rows of one head and walks the keys in
// steps of 32 that its workgroup copies straight into LDS, a ring of three; two
// waves share a SIMD, of workgroups of their own.  S^T = K Q^T leaves lane L with
// row L % 32 of its wave and half of the keys; rounded to 16 bits those registers
// are the second product's B operand as they stand, because the order of keys
// inside a K step is free as long as V^T (transposed LDS reads) takes them in the
// same order.  Softmax statistics never leave the wave, and the only barrier is
// the one that turns the ring.  Probabilities enter the second product in the 16
// bits that its instruction takes (their fp32 sum is taken before): bf16 outputs
// then are off by 2.3e-3 of their size, 1.7e-3 of which is their own rounding.
// Workgroups of 256 rows, whose steps are copied half as often, gain 6% at 16384
// rows and lose 2% at 4 x 4096 and 20% on short ragged prompts; the wide head's
// division of the work (below) loses 15% here.
//
// A call with few tiles divides the keys of each among workgroups that leave
// unnormalised sums, maxima and fp32 partial outputs; join_parts_kernel adds them.
//
// Measured, bf16: 16384 rows, 16 heads: 1.28 ms, 1073 TFLOP/s, against 1223 of a
// large library product; the matrix pipes are busy 56% of the cycles at 1.65 GHz,
// the product's 70% at 1.5 to 1.9.  4 x 4096 rows, 32 heads: 0.76 ms, 908 TFLOP/s,
// 46% at 1.74.  Eight prompts of 36..1023 rows after 129 keys, 64 heads: 167 us for
// 353 MB and 85 GFLOP, 70 us each at the card's rates.  There a tile has 18 steps of 2300 clocks (two workgroups at a
// time; 1280 of them products) and 7 us beside them: finding its place, its
// queries and first keys from HBM, and its output, of which the other
// workgroup of the CU hides about half.
#include "dev_attn.h"

namespace coli {
namespace {

using dev::f32x16;
using dev::f32x2;
using dev::f32x4;
using dev::u32x2;
using dev::u32x4;

constexpr int kRows = 128;        // query rows of a tile
constexpr int kStepKeys = 32;
// A call with few tiles divides the keys of each into parts: at least four steps
// each (with sixteen, 64 rows of 1024 keys and 8 heads take 21 us instead of
// 14.5; undivided they take 29) and at most 64 parts (20 rows of 60000 keys, one
// head: 64 parts 58 us, 32 65 us, 128 75 us: the join reads them one after the other).
constexpr int kLeastSteps = 4;
constexpr int64_t kMostParts = 64;
constexpr int kBlockBytes = kStepKeys * 128;
constexpr int kRing = 4;          // of the wide head, whose values are read a step later
constexpr float kSlack = 8.0f;    // see latent_decode.hip
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr int kSlots = 3;         // ring of the narrow head: steps t, t + 1 and t + 2
constexpr int kAhead = 4;         // LDS reads in flight ahead of the products that use them

// The widths of one head, in 64-column blocks of the LDS step.
template <int NOPE, int V>
struct Head {
    static constexpr int kKeyBlocks = (NOPE + kRope) / 64, kNopeBlocks = NOPE / 64, kValueBlocks = V / 64;
    static constexpr int kDepth = (NOPE + kRope) / 16;          // K steps of the first product
    static constexpr int kBlocks = kKeyBlocks + kValueBlocks;
    static constexpr int kStepBytes = kBlocks * kBlockBytes;
    static constexpr int kQueryBytes = kKeyBlocks * kBlockBytes;   // 32 rows
};

// One row tile of one head.
struct Tile {
    int q0, k0, nk;            // first query token and key of the sequence, its keys
    int head, row0, rows;      // rows row0 .. row0 + rows - 1 of the sequence's queries
    int ahead;                 // row i sees keys up to i + ahead (causal)
    int steps;
    int pieces, slot;          // parts the tile's keys are divided into; this one's place in the scratch
};

// The keys a row of the tile sees (the first `seen` ones).
__device__ __forceinline__ int seen_by(const PromptArgs &a, const Tile &t, int row) {
    return a.causal ? min(t.nk, t.row0 + row + t.ahead + 1) : t.nk;
}

// The wave's 32 rows of queries by way of `at` in LDS, 128 bytes of a row at a
// time; loaded as the products take them, 32 bytes of 32 rows at a time, they
// hold the first step up (64 rows of 1024 keys, 8 heads: 14.7 us, so 13.8; four
// wide prompts of 4096 rows, 32 heads: 1231 and 1220).  After copy_queries(), when
// its copies have landed, read_queries().
template <int DEPTH>
__device__ __forceinline__ void copy_queries(const PromptArgs &a, const Tile &tile, int row0, uint32_t at) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 8 * j + (lane >> 3);
        const int64_t row = tile.q0 + tile.row0 + min(row0 + r, tile.rows - 1);
        const uint8_t *src = a.q + (row * a.q_tok + tile.head * a.q_head) * 2 + (((lane & 7) ^ dev::tile_swz(r)) << 4);
#pragma unroll
        for (int b = 0; b < DEPTH / 4; ++b) dev::copy16_to_lds_free(src + b * 128, at + b * kBlockBytes + j * 1024);
    }
}
template <int DEPTH>
__device__ __forceinline__ void read_queries(const uint8_t *at, u32x4 (&q)[DEPTH]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < DEPTH; ++k)
        q[k] = *reinterpret_cast<const u32x4 *>(at + (k >> 2) * kBlockBytes + dev::tile_unit(lane & 31, 2 * (k & 3) + (lane >> 5)));
}

// Attention of the wave's 32 rows over all steps.  CAREFUL: keys that a row does
// not see have weight zero, and zero times inf or NaN must not reach it; values
// that are not finite are taken as zero where a step hides keys, and a second
// product counts, per output, those that the row does see, which make that
// output NaN.
template <bool BF, int NOPE, int V, bool CAREFUL>
__device__ __forceinline__ void attend(const PromptArgs &a, const Tile &tile, uint8_t *s_kv, uint32_t kv_lds, f32x16 (&acc)[V / 32],
                                       float &m, float &l) {
    using H = Head<NOPE, V>;
    const int lane = threadIdx.x & 63, wave = dev::wave_id(), l31 = lane & 31, lh = lane >> 5;
    const float c = a.scale * kLog2e;
    const int row = 32 * wave + l31;
    // Keys below `open` are seen by every row of the wave, from `shut` on by none.
    const int open = seen_by(a, tile, 32 * wave), shut = seen_by(a, tile, min(32 * wave + 31, tile.rows - 1));
    const int seen_all = seen_by(a, tile, row);

    // Copies: keys 8 w .. + 7 of a step, a 16-byte unit of every block per lane.
    const int cr = 8 * wave + (lane >> 3), unit = ((lane & 7) ^ dev::tile_swz(cr)) << 4;
    struct Copy {
        const uint8_t *kv, *pe;
        uint32_t dst;
    };
    auto aim = [&](int t) {
        const uint32_t dst = kv_lds + (t % kSlots) * H::kStepBytes + wave * 1024;
        t = min(t, tile.steps - 1);                       // past the end the last step is copied again
        const int64_t key = tile.k0 + min(t * kStepKeys + cr, tile.nk - 1);
        return Copy{a.kv + (key * a.kv_tok + tile.head * a.kv_head) * 2 + unit, a.k_pe + key * a.pe_tok * 2 + unit, dst};
    };
    auto copy = [&](const Copy &x, int b) {
        const uint8_t *src = b < H::kNopeBlocks ? x.kv + b * 128 : b == H::kNopeBlocks ? x.pe : x.kv + (b - 1) * 128;
        dev::copy16_to_lds_free(src, x.dst + b * kBlockBytes);
    };
    auto copy_step = [&](int t) {
        const Copy x = aim(t);
#pragma unroll
        for (int b = 0; b < H::kBlocks; ++b) copy(x, b);
    };

#pragma unroll
    for (int cb = 0; cb < V / 32; ++cb)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[cb][i] = 0.0f;
    m = -__builtin_inff();
    l = 0.0f;
    float limit = -__builtin_inff(), offset = 0.0f;       // of a score that calls for a new maximum; of the exponent
    if (tile.steps == 0) return;
    auto key_row = [&](int t, int k) {
        return *reinterpret_cast<const u32x4 *>(s_kv + (t % kSlots) * H::kStepBytes + (k >> 2) * kBlockBytes + dev::tile_unit(l31, 2 * (k & 3) + lh));
    };
    f32x16 s;                                             // scores of step t
    // What follows the scores of a step: the mask, and where a row exceeds its
    // maximum by more than the slack, the new maximum.
    auto largest = [](const f32x16 &x) {
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, x[i]);
        return mx;
    };
    auto settle = [&](int t, float mx) {
        if ((t + 1) * kStepKeys > open) {
            const int seen = seen_all - t * kStepKeys - 4 * lh;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (8 * (i >> 2) + (i & 3) >= seen) s[i] = -__builtin_inff();
            mx = largest(s);
        }
        if (__any(mx > limit)) {
            const float tm = dev::max_halves(mx) * c;
            const float m1 = tm > m + (m == -__builtin_inff() ? 0.0f : kSlack) ? tm : m;
            const float fac = m1 == m ? 1.0f : __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= fac;
            limit = m == -__builtin_inff() ? m : (m + kSlack) / c;
            offset = m == -__builtin_inff() ? 0.0f : -m;
#pragma unroll
            for (int cb = 0; cb < V / 32; ++cb)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[cb][i] *= fac;
        }
    };
    // The queries stand behind the keys of step 1, whose values follow when all
    // waves have read theirs.
    u32x4 q[H::kDepth];
    {
        constexpr int kQueries = H::kStepBytes + H::kKeyBlocks * kBlockBytes;
        copy_queries<H::kDepth>(a, tile, 32 * wave, kv_lds + kQueries + wave * H::kQueryBytes);
        copy_step(0);
        const Copy x = aim(1);
#pragma unroll
        for (int b = 0; b < H::kKeyBlocks; ++b) copy(x, b);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(H::kKeyBlocks) : "memory");
        read_queries<H::kDepth>(s_kv + kQueries + wave * H::kQueryBytes, q);
        dev::lds_barrier();
#pragma unroll
        for (int b = H::kKeyBlocks; b < H::kBlocks; ++b) copy(x, b);
    }
    {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < H::kDepth; ++k) s = dev::mma<BF>(key_row(0, k), q[k], s);
        settle(0, largest(s));
    }
    for (int t = 0; t < tile.steps; ++t) {
        // Step t + 1 has landed, and step t - 1 is read no more.
        dev::copy_barrier();
        if (t * kStepKeys >= shut) {
            copy_step(t + 2);
            continue;
        }
        // The scores of step t + 1 (past the end, of the last step again) are
        // formed while those of step t are weighed and step t + 2 is copied: in
        // four parts of a quarter of each, because the wave stalls at a copy
        // until the CU's address unit takes it (five in a row cost 670 of the
        // step's 2420 clocks) and the products run on meanwhile.
        f32x16 next;
#pragma unroll
        for (int i = 0; i < 16; ++i) next[i] = 0.0f;
        u32x4 kf[kAhead];
        u32x4 p[2];                                       // B operands of the two 16-key products
        constexpr int kPart = H::kDepth / 4;
        const Copy now = aim(t + 2);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);   // over the SIMD's other wave where that one masks and looks for maxima (16384 rows 3.6% faster)
#pragma unroll
        for (int k = 0; k < kAhead; ++k) kf[k] = key_row(t + 1, k);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
#pragma unroll
            for (int k = h * kPart; k < (h + 1) * kPart; ++k) {
                next = dev::mma<BF>(kf[k % kAhead], q[k], next);
                if (k + kAhead < H::kDepth) kf[k % kAhead] = key_row(t + 1, k + kAhead);
            }
#pragma unroll
            for (int j = 2 * h; j < 2 * h + 2; ++j) {
                const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * j], c, offset));
                const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * j + 1], c, offset));
                l += e0 + e1;
                p[j >> 2][j & 3] = dev::pack2<BF>(e0, e1);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = h * H::kBlocks / 4; b < (h + 1) * H::kBlocks / 4; ++b) copy(now, b);
            __builtin_amdgcn_sched_barrier(0);
        }
        // O^T: product k takes keys 16 k + 4 lh + 0..3 and 16 k + 8 + 4 lh + 0..3.
        const uint8_t *vt = s_kv + (t % kSlots) * H::kStepBytes + H::kKeyBlocks * kBlockBytes + 8 * (lane & 1);
        const int vr = 4 * lh + ((lane >> 2) & 3);
        auto value = [&](int n) {                         // of product n: 16 keys n / (V / 32), columns 32 (n % (V / 32))
            const int k = n / (V / 32), cb = n % (V / 32);
            const uint8_t *blk = vt + (cb >> 1) * kBlockBytes + 16 * k * 128;
            const int unit = 4 * (cb & 1) + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
            const u32x2 a0 = dev::read_tr(blk + dev::tile_unit(vr, unit));
            const u32x2 a1 = dev::read_tr(blk + dev::tile_unit(vr + 8, unit));
            return u32x4{a0[0], a0[1], a1[0], a1[1]};
        };
        if (CAREFUL && (t + 1) * kStepKeys > open) {
            const int seen = seen_all - t * kStepKeys - 4 * lh;
            const uint32_t one = BF ? 0x3F80u : 0x3C00u;
#pragma unroll
            for (int cb = 0; cb < V / 32; ++cb) {
                f32x16 n;
#pragma unroll
                for (int i = 0; i < 16; ++i) n[i] = 0.0f;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    u32x4 v = value(k * (V / 32) + cb), off, sees;
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const uint32_t x = dev::nonfinite_halves<BF>(v[d]);
                        v[d] &= ~x;
                        off[d] = x & (one | one << 16);
                        const int at = 16 * k + 8 * (d >> 1) + 2 * (d & 1);
                        sees[d] = (at < seen ? one : 0u) | (at + 1 < seen ? one << 16 : 0u);
                    }
                    acc[cb] = dev::mma<BF>(v, p[k], acc[cb]);
                    n = dev::mma<BF>(off, sees, n);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n[i] > 0.0f) acc[cb][i] = __builtin_nanf("");
            }
        } else {
            constexpr int kN = 2 * (V / 32);
            u32x4 vf[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n) vf[n] = value(n);
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                acc[n % (V / 32)] = dev::mma<BF>(vf[n % kAhead], p[n / (V / 32)], acc[n % (V / 32)]);
                if (n + kAhead < kN) vf[n % kAhead] = value(n + kAhead);
            }
            dev::pipeline<2 * kN, 1, 2, 2 * kAhead>();
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
        s = next;
        settle(t + 1, largest(next));
    }
    // The copies past the end land before the ring is used again.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// The place of this workgroup among `total`: those of one XCD (blockIdx % 8)
// follow each other.  Negative where it has none.
__device__ __forceinline__ int place_of(int total) {
    const int share = (total + 7) / 8, xcd = blockIdx.x & 7, i = blockIdx.x >> 3;
    return i < share && xcd * share + i < total ? xcd * share + i : -1;
}

// The row tile of place `slot`, or the part of its keys that the place takes
// where a call has few tiles; false where it has none.  The row tiles of one
// head, which share K and V in an XCD's L2, follow each other; the last tiles,
// which see the most keys, come first.
__device__ __forceinline__ bool find_tile(const PromptArgs &a, int tiles_cap, int slot, Tile &tile) {
    const int lane = threadIdx.x & 63;
    if (slot < 0) return false;
    tile.slot = slot;
    const int lin = slot / a.split, piece = slot - lin * a.split;
    tile.head = lin / tiles_cap;
    const int want = tiles_cap - 1 - (lin - tile.head * tiles_cap);
    // Sequence and row tile number `want` of the call: each lane counts one
    // sequence's tiles.  The scan ends where it finds them, but for the first place,
    // which looks at the bounds of every sequence.
    int number = 0, nq = 0;
    bool found = false, bad_seq = false;
    for (int b0 = 0, done = 0; b0 < a.n_seq && !(found && slot); b0 += 64) {
        const int b = b0 + lane;
        int n = 0, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
        if (b < a.n_seq) {
            q0 = a.q_start[b];
            q1 = a.q_start[b + 1];
            k0 = a.k_start[b];
            k1 = a.k_start[b + 1];
            const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.n_q;
            if (ok) n = (q1 - q0 + kRows - 1) / kRows;
            bad_seq = bad_seq || !ok || k0 < 0 || k1 < k0 || k1 > a.n_k;
        }
        const int cum = dev::running_sum(n);
        const uint64_t hit = found ? 0 : __ballot(done + cum > want);
        if (hit) {
            const int at = __ffsll(static_cast<unsigned long long>(hit)) - 1;
            found = true;
            number = want - done - (__builtin_amdgcn_readlane(cum, at) - __builtin_amdgcn_readlane(n, at));
            tile.q0 = __builtin_amdgcn_readlane(q0, at);
            nq = __builtin_amdgcn_readlane(q1, at) - tile.q0;
            tile.k0 = __builtin_amdgcn_readlane(k0, at);
            tile.nk = __builtin_amdgcn_readlane(k1, at) - tile.k0;
        }
        done += __builtin_amdgcn_readlane(cum, 63);
    }
    dev::flag_if(bad_seq, a.err, kErrSeq);
    if (!found) return false;
    if (tile.k0 < 0 || tile.nk < 0 || tile.nk > a.n_k - tile.k0) {
        dev::flag_if(threadIdx.x == 0, a.err, kErrSeq);
        tile.k0 = tile.nk = 0;
    }
    tile.row0 = number * kRows;
    tile.rows = min(kRows, nq - tile.row0);
    tile.ahead = tile.nk - nq;
    const int last = seen_by(a, tile, tile.rows - 1);
    tile.steps = last > 0 ? (last + kStepKeys - 1) / kStepKeys : 0;
    // A part is a tile whose sequence begins at the part's first key.
    tile.pieces = min(a.split, max(1, tile.steps / kLeastSteps));
    if (piece >= tile.pieces) return false;
    const int t0 = piece * tile.steps / tile.pieces, t1 = (piece + 1) * tile.steps / tile.pieces;
    tile.k0 += t0 * kStepKeys;
    tile.nk -= t0 * kStepKeys;
    tile.ahead -= t0 * kStepKeys;
    tile.steps = t1 - t0;
    return true;
}

// Partial outputs of a part: block b (32 columns of 32 rows) as its registers
// hold it, four to a store, 256 threads.
template <int V>
__device__ __forceinline__ float *part_of(const PromptArgs &a, int slot, int block) {
    return a.part + (static_cast<int64_t>(slot) * (V / 32) + block) * (16 * 256) + (threadIdx.x & 255) * 4;
}
template <int V>
__device__ __forceinline__ void store_part(const PromptArgs &a, int slot, int block, const f32x16 &acc) {
    float *at = part_of<V>(a, slot, block);
#pragma unroll
    for (int g = 0; g < 4; ++g) *reinterpret_cast<f32x4 *>(at + g * 1024) = f32x4{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
}

// Tiles whose keys were divided: out = sum_i f_i O_i / sum_i f_i l_i with
// f_i = 2^(m_i - max m).  A workgroup joins one block of a tile; its threads
// stand where those that stored the parts stood.
template <bool BF, int V, bool WIDE>
__global__ __launch_bounds__(256) void join_parts_kernel(PromptArgs a, int tiles_cap) {
    Tile tile;
    const int place = place_of(a.n_heads * tiles_cap);
    if (!find_tile(a, tiles_cap, place < 0 ? place : place * a.split, tile) || tile.pieces == 1) return;
    const int wave = dev::wave_id(), l31 = threadIdx.x & 31, lh = (threadIdx.x & 63) >> 5, block = blockIdx.y;
    const int row = WIDE ? 32 * (block & 3) + l31 : 32 * wave + l31;
    const int col = WIDE ? wave * (V / 4) + 32 * (block >> 2) : 32 * block;
    // Four parts' loads are in flight at a time.
    constexpr int kBatch = 4;
    const f32x2 *ml = reinterpret_cast<const f32x2 *>(a.part_ml) + static_cast<int64_t>(tile.slot) * kRows + row;
    const int last = tile.pieces - 1;
    float m = -__builtin_inff(), l = 0.0f;
    for (int i = 0; i < tile.pieces; i += 2 * kBatch) {
        float mi[2 * kBatch];
#pragma unroll
        for (int j = 0; j < 2 * kBatch; ++j) mi[j] = ml[min(i + j, last) * kRows][0];
#pragma unroll
        for (int j = 0; j < 2 * kBatch; ++j) m = fmaxf(m, mi[j]);
    }
    f32x16 acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    for (int i = 0; i < tile.pieces; i += kBatch) {
        f32x2 mli[kBatch];
        f32x4 x[kBatch][4];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int p = min(i + j, last);
            const float *at = part_of<V>(a, tile.slot + p, block);
            mli[j] = ml[p * kRows];
#pragma unroll
            for (int g = 0; g < 4; ++g) x[j][g] = *reinterpret_cast<const f32x4 *>(at + g * 1024);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (i + j > last) break;
            const float f = mli[j][0] == m ? 1.0f : __builtin_amdgcn_exp2f(mli[j][0] - m);
            l = __builtin_fmaf(f, mli[j][1], l);
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[k] = __builtin_fmaf(f, x[j][k >> 2][k & 3], acc[k]);
        }
    }
    const int64_t out_row = static_cast<int64_t>(tile.q0 + tile.row0 + row) * a.n_heads + tile.head;
    dev::store_tile16<BF>(acc, l == 0.0f ? 0.0f : 1.0f / l, row < tile.rows ? a.out + (out_row * V + col) * 2 : nullptr);
    if (a.lse && block == (WIDE ? block & 3 : 0) && lh == 0 && (!WIDE || wave == 0) && row < tile.rows)
        a.lse[out_row] = l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <bool BF, int NOPE, int V>
__global__ __launch_bounds__(256, 2) void latent_prompt_kernel(PromptArgs a, int tiles_cap) {
    // The ring, or steps 0 and 1 without the values of step 1 and the queries:
    // half of a CU's 160 KB for the narrow head.
    using H = Head<NOPE, V>;
    constexpr int kStart = H::kStepBytes + H::kKeyBlocks * kBlockBytes + 4 * H::kQueryBytes;
    __shared__ __align__(1024) uint8_t s_kv[kStart > kSlots * H::kStepBytes ? kStart : kSlots * H::kStepBytes];
    const int tid = threadIdx.x, lane = tid & 63, wave = dev::wave_id();
    const int l31 = lane & 31, lh = lane >> 5;
    const uint32_t kv_lds = dev::lds_address(s_kv);
    Tile tile;
    if (!find_tile(a, tiles_cap, place_of(a.n_heads * tiles_cap * a.split), tile)) return;

    f32x16 acc[V / 32];                                   // [32 columns][32 rows] blocks of O^T
    float m, l;
    attend<BF, NOPE, V, false>(a, tile, s_kv, kv_lds, acc, m, l);
    // Anything that is not finite: again with care, if a step hides keys.
    float z = 0.0f;
#pragma unroll
    for (int cb = 0; cb < V / 32; ++cb)
#pragma unroll
        for (int i = 0; i < 16; ++i) z = __builtin_fmaf(acc[cb][i], 0.0f, z);
    dev::lds_barrier();
    int *bad = reinterpret_cast<int *>(s_kv);             // one per wave
    const bool mine = __any(z != 0.0f);
    if (lane == 0) bad[wave] = mine;
    dev::lds_barrier();
    const bool again = bad[0] | bad[1] | bad[2] | bad[3];
    dev::lds_barrier();
    if (again) {
        attend<BF, NOPE, V, true>(a, tile, s_kv, kv_lds, acc, m, l);
        dev::lds_barrier();                               // the ring is read no more
    }

    const int row = 32 * wave + l31;
    l = dev::sum_halves(l);
    if (tile.pieces > 1) {
#pragma unroll
        for (int cb = 0; cb < V / 32; ++cb) store_part<V>(a, tile.slot, cb, acc[cb]);
        if (lh == 0) *reinterpret_cast<f32x2 *>(a.part_ml + (static_cast<int64_t>(tile.slot) * kRows + row) * 2) = f32x2{m, l};
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t first = static_cast<int64_t>(tile.q0 + tile.row0 + 32 * wave) * a.n_heads + tile.head;
#pragma unroll
    for (int cb = 0; cb < V / 32; cb += 2)
        dev::store_rows16<BF>(acc[cb], acc[cb + 1], inv, s_kv + 1024 + wave * kBlockBytes, a.out + first * V * 2 + 64 * cb,
                              static_cast<int64_t>(a.n_heads) * V * 2, tile.rows - 32 * wave);
    if (a.lse && lh == 0 && row < tile.rows)
        a.lse[first + static_cast<int64_t>(l31) * a.n_heads] = l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// ---- The wide head: scoring and summing waves ------------------------------
//
// A wave with 32 rows of queries (64 registers) and of outputs (128) leaves too
// little of its 256 registers to the fragments in flight.  The wide head
// therefore divides the work by kind, as latent_decode.hip does: 128 rows a
// workgroup; four scoring waves with 32 rows each write the 16-bit
// probabilities of step t to LDS, four summing waves with a quarter of the
// value columns each add step t - 1 for all rows and copy step t + 2.  Each
// SIMD holds one of either kind.  (One kind of wave, 64-key tiles: 281 spilled
// registers, 7.8 ms for 4 x 4096 rows, 32 heads, f16; so 1.25 ms, 881 TFLOP/s of
// 1164 of a large library product, the matrix pipes busy 43% at 1.76 GHz.)  A row's scores lie in one wave, which moves
// its maximum by itself and leaves the rows' factors for the summing waves.
constexpr int kSplitThreads = 512;

__device__ __forceinline__ int weight_unit(int r, int q) { return r * 64 + ((q ^ ((r >> 2) & 3)) << 4); }

struct Shared {
    uint8_t *kv, *p;           // [kRing] steps of keys and values; [2] steps of probabilities
    float *fac, *sum;          // [2][128] factors by step parity; [128] row sums
    int *raise;                // [3][4] by step and scoring wave: factors to apply
};

template <bool BF, int NOPE, int V>
__device__ __forceinline__ void score_rows(const PromptArgs &a, const Tile &tile, const Shared &sh, float &m) {
    using H = Head<NOPE, V>;
    const int lane = threadIdx.x & 63, wave = dev::wave_id(), l31 = lane & 31, lh = lane >> 5;
    const float c = a.scale * kLog2e;
    const int row = 32 * wave + l31;
    // Keys below `open` are seen by every row of the wave, from `shut` on by none.
    const int open = seen_by(a, tile, 32 * wave);
    const int shut = 32 * wave < tile.rows ? seen_by(a, tile, min(32 * wave + 31, tile.rows - 1)) : 0;
    const int seen_all = seen_by(a, tile, row);
    // The queries stand where steps 2 and 3 are copied to after the first barrier.
    u32x4 q[H::kDepth];
    static_assert(4 * H::kQueryBytes <= 2 * H::kStepBytes);
    copy_queries<H::kDepth>(a, tile, 32 * wave, dev::lds_address(sh.kv) + 2 * H::kStepBytes + wave * H::kQueryBytes);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    read_queries<H::kDepth>(sh.kv + 2 * H::kStepBytes + wave * H::kQueryBytes, q);
    __builtin_amdgcn_s_setprio(2);   // the step waits for these waves: the summing ones fill what they leave
    m = -__builtin_inff();
    float l = 0.0f, limit = -__builtin_inff(), offset = 0.0f;
    for (int t = 0; t < tile.steps; ++t) {
        dev::lds_barrier();
        if (lane == 0) sh.raise[((t + 1) % 3) * 4 + wave] = 0;
        uint8_t *pw = sh.p + (t & 1) * (kRows * 64);
        if (t * kStepKeys >= shut) {
#pragma unroll
            for (int g = 0; g < 4; ++g) *reinterpret_cast<u32x2 *>(pw + weight_unit(row, g) + 8 * lh) = u32x2{0, 0};
            continue;
        }
        const uint8_t *kv = sh.kv + (t & (kRing - 1)) * H::kStepBytes;
        auto key = [&](int k) { return *reinterpret_cast<const u32x4 *>(kv + (k >> 2) * kBlockBytes + dev::tile_unit(l31, 2 * (k & 3) + lh)); };
        f32x16 s[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) s[0][i] = s[1][i] = 0.0f;
        u32x4 kf[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) kf[k] = key(k);
#pragma unroll
        for (int k = 0; k < H::kDepth; ++k) {
            s[k & 1] = dev::mma<BF>(kf[k % 6], q[k], s[k & 1]);
            if (k + 6 < H::kDepth) kf[k % 6] = key(k + 6);
        }
        dev::pipeline<H::kDepth, 1, 1, 6>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[0][i] += s[1][i];
        if ((t + 1) * kStepKeys > open) {
            const int seen = seen_all - t * kStepKeys - 4 * lh;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (8 * (i >> 2) + (i & 3) >= seen) s[0][i] = -__builtin_inff();
        }
        float mx = s[0][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[0][i]);
        if (__any(mx > limit)) {
            const float tm = dev::max_halves(mx) * c;
            const float m1 = tm > m + (m == -__builtin_inff() ? 0.0f : kSlack) ? tm : m;
            const float fac = m1 == m ? 1.0f : __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= fac;
            limit = m == -__builtin_inff() ? m : (m + kSlack) / c;
            offset = m == -__builtin_inff() ? 0.0f : -m;
            if (lh == 0) sh.fac[(t & 1) * kRows + row] = fac;
            if (lane == 0) sh.raise[(t % 3) * 4 + wave] = 1;
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[0][4 * g + j], c, offset));
            l += (e[0] + e[1]) + (e[2] + e[3]);
            *reinterpret_cast<u32x2 *>(pw + weight_unit(row, g) + 8 * lh) =
                u32x2{dev::pack2<BF>(e[0], e[1]), dev::pack2<BF>(e[2], e[3])};
        }
    }
    l = dev::sum_halves(l);
    if (lh == 0) sh.sum[row] = l;
    if (tile.steps) dev::lds_barrier();                   // the last step's probabilities
}

// Columns (V / 4) w .. of the summing wave w, all rows.  CAREFUL as in attend().
template <bool BF, int NOPE, int V, bool CAREFUL>
__device__ __forceinline__ bool sum_columns(const PromptArgs &a, const Tile &tile, const Shared &sh, uint32_t kv_lds, f32x16 (&acc)[V / 128][4]) {
    using H = Head<NOPE, V>;
    constexpr int kCols = V / 128;                        // 32-column blocks of the wave
    const int lane = threadIdx.x & 63, wave = dev::wave_id() & 3, l31 = lane & 31, lh = lane >> 5;
#pragma unroll
    for (int cb = 0; cb < kCols; ++cb)
#pragma unroll
        for (int rb = 0; rb < 4; ++rb)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[cb][rb][i] = 0.0f;
    if (tile.steps == 0) return false;

    // Copies: keys 8 w .. + 7 of a step, a 16-byte unit of every block per lane.
    const int cr = 8 * wave + (lane >> 3), unit = ((lane & 7) ^ dev::tile_swz(cr)) << 4;
    struct Copy {
        const uint8_t *kv, *pe;
        uint32_t dst;
    };
    auto aim = [&](int t) {
        t = min(t, tile.steps - 1);                       // past the end the last step is copied again
        const int64_t key = tile.k0 + min(t * kStepKeys + cr, tile.nk - 1);
        return Copy{a.kv + (key * a.kv_tok + tile.head * a.kv_head) * 2 + unit, a.k_pe + key * a.pe_tok * 2 + unit,
                    kv_lds + (t & (kRing - 1)) * H::kStepBytes + wave * 1024};
    };
    auto copy = [&](const Copy &x, int b) {
        const uint8_t *src = b < H::kNopeBlocks ? x.kv + b * 128 : b == H::kNopeBlocks ? x.pe : x.kv + (b - 1) * 128;
        dev::copy16_to_lds_free(src, x.dst + b * kBlockBytes);
    };
    auto copy_all = [&](const Copy &x) {
#pragma unroll
        for (int b = 0; b < H::kBlocks; ++b) copy(x, b);
    };
    const int vr = 8 * lh + ((lane >> 2) & 3);
    auto step = [&](int t, bool more, Copy &now) {
        const u32x4 raise = *reinterpret_cast<const u32x4 *>(sh.raise + (t % 3) * 4);
        const uint8_t *pr = sh.p + (t & 1) * (kRows * 64);
        const uint8_t *vt = sh.kv + (t & (kRing - 1)) * H::kStepBytes + H::kKeyBlocks * kBlockBytes + 8 * (lane & 1);
        u32x4 pf[2][4], vf[2][kCols];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int cb = 0; cb < kCols; ++cb) {
                const int col = wave * kCols + cb;        // 32-column block of the head's values
                const uint8_t *blk = vt + (col >> 1) * kBlockBytes + 16 * k * 128;
                const int u = 4 * (col & 1) + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
                const u32x2 a0 = dev::read_tr(blk + dev::tile_unit(vr, u));
                const u32x2 a1 = dev::read_tr(blk + dev::tile_unit(vr + 4, u));
                vf[k][cb] = u32x4{a0[0], a0[1], a1[0], a1[1]};
            }
#pragma unroll
            for (int rb = 0; rb < 4; ++rb) pf[k][rb] = *reinterpret_cast<const u32x4 *>(pr + weight_unit(32 * rb + l31, 2 * k + lh));
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rb = 0; rb < 4; ++rb)
            if (__builtin_amdgcn_readfirstlane(raise[rb])) {
                const float f = sh.fac[(t & 1) * kRows + 32 * rb + l31];
#pragma unroll
                for (int cb = 0; cb < kCols; ++cb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[cb][rb][i] *= f;
            }
        if (CAREFUL && (t + 1) * kStepKeys > seen_by(a, tile, 0)) {
            const uint32_t one = BF ? 0x3F80u : 0x3C00u;
#pragma unroll
            for (int cb = 0; cb < kCols; ++cb)
#pragma unroll
                for (int rb = 0; rb < 4; ++rb) {
                    const int seen = seen_by(a, tile, 32 * rb + l31) - t * kStepKeys - 8 * lh;
                    f32x16 n;
#pragma unroll
                    for (int i = 0; i < 16; ++i) n[i] = 0.0f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        u32x4 v = vf[k][cb], off, sees;
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const uint32_t x = dev::nonfinite_halves<BF>(v[d]);
                            v[d] &= ~x;
                            off[d] = x & (one | one << 16);
                            const int at = 16 * k + 2 * d;
                            sees[d] = (at < seen ? one : 0u) | (at + 1 < seen ? one << 16 : 0u);
                        }
                        acc[cb][rb] = dev::mma<BF>(v, pf[k][rb], acc[cb][rb]);
                        n = dev::mma<BF>(off, sees, n);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (n[i] > 0.0f) acc[cb][rb][i] = __builtin_nanf("");
                }
            if (more) copy_all(now);
        } else {
            // The copies are issued between the products.
            int b = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int cb = 0; cb < kCols; ++cb)
#pragma unroll
                    for (int rb = 0; rb < 4; rb += 2) {
                        __builtin_amdgcn_sched_barrier(0);
                        if (more && b < H::kBlocks) copy(now, b++);
                        __builtin_amdgcn_sched_barrier(0);
                        acc[cb][rb] = dev::mma<BF>(vf[k][cb], pf[k][rb], acc[cb][rb]);
                        acc[cb][rb + 1] = dev::mma<BF>(vf[k][cb], pf[k][rb + 1], acc[cb][rb + 1]);
                    }
            __builtin_amdgcn_sched_barrier(0);
            if (more)
#pragma unroll
                for (; b < H::kBlocks; ++b) copy(now, b);
        }
        if (more) now = aim(t + 4);
    };

    copy_all(aim(0));
    copy_all(aim(1));
    Copy now = aim(2);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(H::kBlocks) : "memory");
    dev::lds_barrier();
    copy_all(now);
    now = aim(3);
    for (int t = 1; t < tile.steps; ++t) {
        // Step t has landed when only the copies of step t + 1 are in flight.
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(H::kBlocks) : "memory");
        dev::lds_barrier();
        step(t - 1, true, now);
    }
    dev::copy_barrier();
    step(tile.steps - 1, false, now);
    float z = 0.0f;
#pragma unroll
    for (int cb = 0; cb < kCols; ++cb)
#pragma unroll
        for (int rb = 0; rb < 4; ++rb)
#pragma unroll
            for (int i = 0; i < 16; ++i) z = __builtin_fmaf(acc[cb][rb][i], 0.0f, z);
    return __any(z != 0.0f);
}

template <bool BF, int NOPE, int V>
__global__ __launch_bounds__(kSplitThreads, 2) void latent_prompt_split_kernel(PromptArgs a, int tiles_cap) {
    __shared__ __align__(1024) uint8_t s_kv[kRing * Head<NOPE, V>::kStepBytes];
    __shared__ __align__(1024) uint8_t s_p[2 * kRows * 64];
    __shared__ float s_fac[2 * kRows], s_sum[kRows];
    __shared__ __align__(16) int s_raise[12];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = dev::wave_id();
    const int l31 = lane & 31;
    const uint32_t kv_lds = dev::lds_address(s_kv);
    Tile tile;
    if (!find_tile(a, tiles_cap, place_of(a.n_heads * tiles_cap * a.split), tile)) return;
    const Shared sh{s_kv, s_p, s_fac, s_sum, s_raise};
    const int64_t first = static_cast<int64_t>(tile.q0 + tile.row0) * a.n_heads + tile.head;
    if (tid == 0) s_bad = 0;
    if (tid < 12) s_raise[tid] = 0;
    dev::lds_barrier();
    if (wave < 4) {
        float m;
        score_rows<BF, NOPE, V>(a, tile, sh, m);
        dev::lds_barrier();
        if (s_bad) {                                      // the same scores again for the careful sums
            dev::lds_barrier();
            score_rows<BF, NOPE, V>(a, tile, sh, m);
            dev::lds_barrier();
        }
        const int row = 32 * wave + l31;
        const float l = s_sum[row];
        if (tile.pieces > 1) {
            if (lane < 32) *reinterpret_cast<f32x2 *>(a.part_ml + (static_cast<int64_t>(tile.slot) * kRows + row) * 2) = f32x2{m, l};
            return;
        }
        if (a.lse && lane < 32 && row < tile.rows)
            a.lse[first + static_cast<int64_t>(row) * a.n_heads] = l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
    } else {
        f32x16 acc[V / 128][4];                           // [32 columns][32 rows] blocks of O^T
        if (sum_columns<BF, NOPE, V, false>(a, tile, sh, kv_lds, acc)) s_bad = 1;
        dev::lds_barrier();
        if (s_bad) {
            if (lane < 12) s_raise[lane] = 0;
            dev::lds_barrier();
            sum_columns<BF, NOPE, V, true>(a, tile, sh, kv_lds, acc);
            dev::lds_barrier();
        }
        if (tile.pieces > 1) {
#pragma unroll
            for (int cb = 0; cb < V / 128; ++cb)
#pragma unroll
                for (int rb = 0; rb < 4; ++rb) store_part<V>(a, tile.slot, 4 * cb + rb, acc[cb][rb]);
            return;
        }
#pragma unroll
        for (int rb = 0; rb < 4; ++rb) {
            const int row = 32 * rb + l31;
            const float l = s_sum[row], inv = l == 0.0f ? 0.0f : 1.0f / l;
            static_assert(V == 256);                      // two blocks of columns a wave
            dev::store_rows16<BF>(acc[0][rb], acc[1][rb], inv, s_kv + (wave & 3) * kBlockBytes,
                                  a.out + ((first + 32ll * rb * a.n_heads) * V + (wave & 3) * (V / 4)) * 2,
                                  static_cast<int64_t>(a.n_heads) * V * 2, tile.rows - 32 * rb);
        }
    }
}

// Row tiles of a call, an upper bound (every sequence may end in a part of
// one), and the workgroups for them, a multiple of the XCDs.  A call with fewer
// tiles than the chip holds workgroups divides the keys of each.
template <typename K, typename J>
hipError_t launch_tiles(PromptArgs &a, K kernel, J join, int threads, int blocks, int places, hipStream_t s) {
    const int64_t seqs = std::min(a.n_seq, a.n_q), cap = (a.n_q - seqs) / kRows + seqs, tiles = cap * a.n_heads;
    const int64_t most = (a.n_k + kStepKeys - 1) / kStepKeys / kLeastSteps;
    // Without much context the first tiles see few keys and the last most: two
    // rounds of parts even that out, where they are of 24 steps or more (4096
    // rows, 12 narrow heads: 127 us in one round, 110 in two; 6 wide heads 114 and 84;
    // but 1024 rows, 32 narrow heads: 34 and 39).
    const int64_t even = a.causal && a.n_k < 2ll * a.n_q ? std::min<int64_t>(2 * places, a.part_cap) / tiles : 0;
    const int64_t want = std::max<int64_t>(std::min(places, a.part_cap) / tiles, std::min<int64_t>(even, a.n_k / a.n_seq / (24 * kStepKeys)));
    a.split = static_cast<int>(std::max<int64_t>(1, std::min({want, most, kMostParts})));
    const int64_t grid = (tiles * a.split + 7) / 8 * 8;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    launch(kernel, static_cast<unsigned>(grid), threads, 0, s, a, static_cast<int>(cap));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.split == 1) return e;
    launch(join, dim3(static_cast<unsigned>((tiles + 7) / 8 * 8), blocks), 256, 0, s, a, static_cast<int>(cap));
    return hipGetLastError();
}

template <bool BF>
hipError_t launch_typed(PromptArgs &a, int nope, int n_cu, hipStream_t s) {
    if (nope == 192)
        return launch_tiles(a, latent_prompt_split_kernel<BF, 192, 256>, join_parts_kernel<BF, 256, true>, kSplitThreads, 256 / 32, n_cu, s);
    return launch_tiles(a, latent_prompt_kernel<BF, 128, 128>, join_parts_kernel<BF, 128, false>, 256, 128 / 32, 2 * n_cu, s);
}

}  // namespace

hipError_t launch_latent_prompt(PromptArgs a, bool bf16, int nope, int n_cu, hipStream_t s) {
    return bf16 ? launch_typed<true>(a, nope, n_cu, s) : launch_typed<false>(a, nope, n_cu, s);
}

}  // namespace coli
