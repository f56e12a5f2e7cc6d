// latent_prompt.hip -- expanded latent attention of whole prompts: per-head
// keys and values from the up-projection, one rotary key shared by the heads.
//
//   s_j = scale (q_nope . k_j + q_pe . r_j),  o = sum_j softmax(s)_j v_j,
// causal with the queries as the last tokens of their sequence.  k_j and v_j
// are read where the up-projection left them ([token][head][nope + v]) and the
// rotary part from its own rows, so no key is ever assembled in memory.
//
// A 512-thread workgroup (two waves per SIMD) takes 256 query rows of one head,
// 32 per wave, and walks 64-key tiles that are copied straight into LDS,
// double buffered.  S^T = K Q^T leaves lane L with row L % 32 of its wave and
// half of the keys; rounded to 16 bits those registers are the second
// product's B operand as they stand, because the order of keys inside a K step
// is free as long as V^T (transposed LDS reads) takes them in the same order.
// Softmax statistics never leave the wave, and the only barrier is the one
// that turns the buffers.
#include "dev_attn.h"

namespace coli {
namespace {

using dev::f32x16;
using dev::u32x2;
using dev::u32x4;

constexpr int kBlockBytes = kTileKeys * 128;
constexpr float kSlack = 8.0f;    // see latent_decode.hip
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves;

template <bool BF, int NOPE, int V>
__global__ __launch_bounds__(64 * kWaves, 2) void latent_prompt_kernel(PromptArgs a, int tiles_cap) {
    constexpr int kKeyBlocks = (NOPE + kRope) / 64, kNopeBlocks = NOPE / 64, kValueBlocks = V / 64;
    constexpr int kSteps = (NOPE + kRope) / 16, kBlocks = kKeyBlocks + kValueBlocks;
    constexpr int kTileBytes = kBlocks * kBlockBytes;
    __shared__ __align__(1024) uint8_t s_kv[2 * kTileBytes];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = dev::wave_id();
    const int l31 = lane & 31, lh = lane >> 5;
    const uint32_t kv_lds = dev::lds_address(s_kv);
    const float c = a.scale * kLog2e;

    // Workgroups of one XCD (blockIdx % 8) take the row tiles of the same
    // heads, which share K and V in its L2; the last tiles, which see the most
    // keys, come first.
    const int total = a.n_heads * tiles_cap, share = (total + 7) / 8;
    const int lin = static_cast<int>(blockIdx.x & 7) * share + static_cast<int>(blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= share || lin >= total) return;
    const int head = lin / tiles_cap, want = tiles_cap - 1 - (lin - head * tiles_cap);

    // Sequence and row tile number `want` of the call: each lane counts one
    // sequence's tiles.
    int seq = -1, tile = 0;
    bool bad_seq = false;
    for (int b0 = 0, done = 0; b0 < a.n_seq; b0 += 64) {
        const int b = b0 + lane;
        int n = 0;
        if (b < a.n_seq) {
            const int q0 = a.q_start[b], q1 = a.q_start[b + 1];
            if (q0 >= 0 && q1 >= q0 && q1 <= a.n_q) n = (q1 - q0 + kRows - 1) / kRows;
            else bad_seq = true;
        }
        int cum = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(cum, o, 64);
            if (lane >= o) cum += y;
        }
        const uint64_t hit = __ballot(done + cum > want);
        if (hit) {
            const int at = __ffsll(static_cast<unsigned long long>(hit)) - 1;
            seq = b0 + at;
            tile = want - done - (__shfl(cum, at, 64) - __shfl(n, at, 64));
            break;
        }
        done += __shfl(cum, 63, 64);
    }
    dev::flag_if(bad_seq, a.err, kErrSeq);
    seq = __builtin_amdgcn_readfirstlane(seq);
    tile = __builtin_amdgcn_readfirstlane(tile);
    if (seq < 0) return;
    const int q0 = a.q_start[seq], nq = a.q_start[seq + 1] - q0;
    int k0 = a.k_start[seq], nk = a.k_start[seq + 1] - k0;
    if (k0 < 0 || nk < 0 || nk > a.n_k - k0) {
        dev::flag_if(tid == 0, a.err, kErrSeq);
        k0 = nk = 0;
    }
    const int row0 = tile * kRows, rows = min(kRows, nq - row0);
    const int row = 32 * wave + l31, qrow = row0 + min(row, rows - 1);
    const int ahead = nk - nq;                            // row i sees keys up to i + ahead
    const int last = a.causal ? min(nk, row0 + rows + ahead) : nk;
    const int n_tiles = last > 0 ? (last + kTileKeys - 1) / kTileKeys : 0;
    // Keys below `open` are seen by every row of the wave; keys from `shut` on
    // by none.
    const int open = a.causal ? min(nk, row0 + 32 * wave + ahead + 1) : nk;
    const int shut = a.causal ? min(nk, row0 + min(32 * wave + 32, rows) + ahead) : nk;

    u32x4 q[kSteps];
    {
        const uint8_t *src = a.q + (static_cast<int64_t>(q0 + qrow) * a.q_tok + head * a.q_head) * 2 + 16 * lh;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) q[k] = dev::gload<u32x4>(src + 32 * k);
    }

    // Copies: each wave fetches eight keys, a 16-byte unit per lane and block.
    const int cr = 8 * wave + (lane >> 3);
    const int cu = ((lane & 7) ^ dev::tile_swz(cr)) << 4;
    auto copy_tile = [&](int t, int buf) {
        const int64_t key = k0 + min(t * kTileKeys + cr, nk - 1);
        const uint8_t *src = a.kv + (key * a.kv_tok + head * a.kv_head) * 2 + cu;
        const uint8_t *pe = a.k_pe + key * a.pe_tok * 2 + cu;
        const uint32_t dst = kv_lds + buf * kTileBytes + wave * 1024;
#pragma unroll
        for (int b = 0; b < kNopeBlocks; ++b) dev::copy16_to_lds(src + b * 128, dst + b * kBlockBytes);
        dev::copy16_to_lds(pe, dst + kNopeBlocks * kBlockBytes);
#pragma unroll
        for (int b = 0; b < kValueBlocks; ++b)
            dev::copy16_to_lds(src + (kNopeBlocks + b) * 128, dst + (kKeyBlocks + b) * kBlockBytes);
    };

    f32x16 acc[V / 32];                                   // [32 columns][32 rows] blocks of O^T
    float m, l;
    for (int careful = 0; careful < 2; ++careful) {
#pragma unroll
        for (int cb = 0; cb < V / 32; ++cb)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[cb][i] = 0.0f;
        m = -__builtin_inff();
        l = 0.0f;
        dev::lds_barrier();                               // the buffers of the pass before are free
        if (tid == 0) s_bad = 0;
        if (n_tiles) copy_tile(0, 0);
        for (int t = 0; t < n_tiles; ++t) {
            const int buf = t & 1;
            const uint8_t *kv = s_kv + buf * kTileBytes;
            dev::copy_barrier();
            if (t + 1 < n_tiles) copy_tile(t + 1, buf ^ 1);
            if (t * kTileKeys >= shut) continue;
            f32x16 s[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[kb][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const uint8_t *blk = kv + (k >> 2) * kBlockBytes;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    const u32x4 kf = *reinterpret_cast<const u32x4 *>(blk + kb * 32 * 128 + dev::tile_unit(l31, 2 * (k & 3) + lh));
                    s[kb] = dev::mma<BF>(kf, q[k], s[kb]);
                }
            }
            const bool masked = (t + 1) * kTileKeys > open;
            if (masked) {
                const int seen = (a.causal ? min(nk, row0 + row + ahead + 1) : nk) - t * kTileKeys - 4 * lh;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (32 * kb + 8 * (i >> 2) + (i & 3) >= seen) s[kb][i] = -__builtin_inff();
            }
            float mx = s[0][0];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[kb][i]);
            mx = dev::max_halves(mx);
            const float tm = mx * c;
            const float m1 = tm > m + kSlack ? tm : m;
            if (__any(m1 != m)) {
                const float fac = m1 == m ? 1.0f : __builtin_amdgcn_exp2f(m - m1);
                l *= fac;
#pragma unroll
                for (int cb = 0; cb < V / 32; ++cb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[cb][i] *= fac;
                m = m1;
            }
            const float ms = m1 == -__builtin_inff() ? 0.0f : m1;
            u32x4 p[4];                                   // B operands of the four 16-key steps
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][2 * j], c, -ms));
                    const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][2 * j + 1], c, -ms));
                    l += e0 + e1;
                    p[2 * kb + (j >> 2)][j & 3] = dev::pack2<BF>(e0, e1);
                }
            // O^T: step k takes keys 16 k + 4 lh + 0..3 and 16 k + 8 + 4 lh + 0..3.
            const uint8_t *vt = kv + kKeyBlocks * kBlockBytes;
            const int vr = 4 * lh + ((lane >> 2) & 3);
            auto value = [&](int k, int cb) {
                const uint8_t *blk = vt + (cb >> 1) * kBlockBytes + 16 * k * 128 + 8 * (lane & 1);
                const int unit = 4 * (cb & 1) + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
                const u32x2 a0 = dev::read_tr(blk + dev::tile_unit(vr, unit));
                const u32x2 a1 = dev::read_tr(blk + dev::tile_unit(vr + 8, unit));
                return u32x4{a0[0], a0[1], a1[0], a1[1]};
            };
            if (!(careful && masked)) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int cb = 0; cb < V / 32; ++cb) acc[cb] = dev::mma<BF>(value(k, cb), p[k], acc[cb]);
            } else {
                // A hidden key's weight is zero, and zero times inf or NaN must
                // not reach the row: values that are not finite are taken as
                // zero, and a second product counts, per output, those that
                // the row does see, which make that output NaN.
                const int seen = (a.causal ? min(nk, row0 + row + ahead + 1) : nk) - t * kTileKeys - 4 * lh;
                const uint32_t one = BF ? 0x3F80u : 0x3C00u;
#pragma unroll
                for (int cb = 0; cb < V / 32; ++cb) {
                    f32x16 n;
#pragma unroll
                    for (int i = 0; i < 16; ++i) n[i] = 0.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        u32x4 v = value(k, cb), off, sees;
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const uint32_t x = dev::nonfinite_halves<BF>(v[d]);
                            v[d] &= ~x;
                            off[d] = x & (one | one << 16);
                            const int key = 16 * k + 8 * (d >> 1) + 2 * (d & 1);
                            sees[d] = (key < seen ? one : 0u) | (key + 1 < seen ? one << 16 : 0u);
                        }
                        acc[cb] = dev::mma<BF>(v, p[k], acc[cb]);
                        n = dev::mma<BF>(off, sees, n);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (n[i] > 0.0f) acc[cb][i] = __builtin_nanf("");
                }
            }
        }
        float z = 0.0f;
#pragma unroll
        for (int cb = 0; cb < V / 32; ++cb)
#pragma unroll
            for (int i = 0; i < 16; ++i) z = __builtin_fmaf(acc[cb][i], 0.0f, z);
        dev::lds_barrier();
        if (__any(z != 0.0f)) s_bad = 1;
        dev::lds_barrier();
        if (!s_bad) break;
    }

    l = dev::sum_halves(l);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t out_row = static_cast<int64_t>(q0 + row0 + row) * a.n_heads + head;
    uint8_t *o = row < rows ? a.out + out_row * V * 2 : nullptr;
#pragma unroll
    for (int cb = 0; cb < V / 32; ++cb) dev::store_tile16<BF>(acc[cb], inv, o ? o + 64 * cb : nullptr);
    if (a.lse && lh == 0 && row < rows)
        a.lse[out_row] = l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <bool BF>
hipError_t launch_typed(const PromptArgs &a, int nope, unsigned grid, int cap, hipStream_t s) {
    if (nope == 192) launch(latent_prompt_kernel<BF, 192, 256>, grid, 64 * kWaves, 0, s, a, cap);
    else launch(latent_prompt_kernel<BF, 128, 128>, grid, 64 * kWaves, 0, s, a, cap);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_latent_prompt(const PromptArgs &a, bool bf16, int nope, hipStream_t s) {
    // Every sequence may end in a part of a tile: an upper bound of the tiles.
    const int64_t cap = std::min<int64_t>(a.n_q, a.n_q / kRows + a.n_seq);
    const int64_t grid = (cap * a.n_heads + 7) / 8 * 8;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    return bf16 ? launch_typed<true>(a, nope, static_cast<unsigned>(grid), static_cast<int>(cap), s)
                : launch_typed<false>(a, nope, static_cast<unsigned>(grid), static_cast<int>(cap), s);
}

}  // namespace coli
