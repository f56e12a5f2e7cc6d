// beam.hip -- beam search's selection: of all continuations of a group's beams the
// `keep` best ones.
//
// The score of token x behind beam b is S = score_b + z_x - log sum_y exp z_y.
// Within a beam the order of the scores is that of the logits, so a workgroup
// looks at a chunk of one row by itself: it leaves the chunk's maximum and sum of
// exponentials and its `keep` best logits, all from one pass over values that stay
// in registers.  A second launch, a workgroup to a group, joins the sums of
// each row and the lists of all rows, the scores taken in 64 bits: the candidates
// of two beams can lie nearer to each other than the 32-bit roundings of their
// scores.  The sum in a score's logarithm is of fp32 exponentials, added in fp32 within a
// chunk, which keeps beams apart to about 1e-7.  (One launch, the join by each group's last workgroup: 32 groups of 8 beams of
// 151643 logits 77 us, as lists are then handed over past the caches, so 42; one group of
// 4 beams 9.7 and 10.2 us.)
//
// Measured, fp32 logits, keep 16: 32 x 8 x 151643, 155 MB, 36 us and 7 for the join (kernel
// times; both 42 us called in turn), 4.3 TB/s where a plain read reaches 7.2: bound by the
// vector work behind the loads (exponentials, the threshold's and the list's ballots) in 89
// registers, five workgroups a CU, each with one round of loads.  From bf16 or f16 53 us: half the
// bytes, in loads half as wide, and the same work after a conversion.  1 x 4 x 32000,
// keep 8: 5 and 4.6 us, two launches and their latencies.
//
// The best of a chunk: a lane's largest value is known from the pass.  The keep-th
// largest of a wave's 64 lane maxima is a value that keep elements of the wave
// reach; the largest such value of the four waves is a threshold that a few times
// keep elements of the chunk reach, and those are ranked by counting.  Of 8192 normal logits
// 45 to 65 reach it at keep 16, 140 at 32, 290 at 48; at 64, where it is the least of a wave's
// maxima, 700 to 1000, and one chunk in eight has more than are ranked and takes its maxima
// one after the other.  32 x 8 x 151643 so takes 61 us at keep 32, 127 at 48 and 860 at 64.
#include "coli_moe.h"
#include "dev_attn.h"

namespace coli {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kCandidates = 1024;        // elements at or above the threshold that are ranked by counting
constexpr int kJoinThreads = 512, kJoinCandidates = 2048;
constexpr int kHeld = 8;                 // a thread's candidates that stay in registers
constexpr float kLog2e = 1.44269504088896341f;

// The smallest key of a candidate: of -FLT_MAX.
constexpr uint32_t kLeastKey = 0x00800000u;

// Values in the order of their keys: NaN counts as -inf, whose key is zero, no
// candidate; -0 and +0 share a key.
__device__ __forceinline__ uint32_t key_of(float v) { return v > -__builtin_inff() ? dev::float_key(v) : 0u; }
__device__ __forceinline__ float value_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key); }
// A value's key above its beam and token, lower ones first: the lower bits are their
// number's complement.
constexpr int kTokenBits = 20;
__device__ __forceinline__ uint64_t packed(uint32_t key, uint32_t id) { return static_cast<uint64_t>(key) << 32 | static_cast<uint32_t>(~id); }

// The largest key that `keep` lanes of the wave reach (0 where fewer than that have a
// candidate), by its bits from the highest down.  (A key that up to a quarter more lanes
// reach is found sooner, but leaves more to rank: 256 rows of 151643 logits 49 us, so 44.)
__device__ __forceinline__ uint32_t reached(uint32_t key, int keep) {
    uint32_t t = 0;
    for (int b = 31; b >= 0; --b) {
        const uint32_t up = t | 1u << b;
        const int n = __popcll(__ballot(key >= up));
        if (n >= keep) t = up;
        if (n == keep) break;
    }
    return t;
}

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));

// EACH elements per thread, four neighbours at a time.
template <int KIND, int EACH>
__global__ __launch_bounds__(kThreads) void select_kernel(SelectArgs a, int row0, int chunks) {
    constexpr int kGroups = EACH / 4, kChunk = kThreads * EACH;
    __shared__ uint64_t s_cand[kCandidates];
    __shared__ float s_max[kWaves], s_sum[kWaves];
    __shared__ uint32_t s_reach[kWaves];
    __shared__ uint64_t s_top[kWaves];
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 63, wave = dev::wave_id();
    const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks, keep = a.keep;
    const int first = chunk * kChunk;
    constexpr int kSize = KIND == COLI_PROB_F32 ? 4 : 2;
    const uint8_t *z = a.logits + (static_cast<int64_t>(row0) + row) * a.stride * kSize;
    float x[EACH];
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        const int at = first + (j * kThreads + tid) * 4;
        if (at + 4 <= a.vocab) {
            if constexpr (KIND == COLI_PROB_F32) {
                const f32x4u v = __builtin_nontemporal_load(reinterpret_cast<const f32x4u *>(z + 4ll * at));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * j + i] = v[i];
            } else {
                const u16x4u v = __builtin_nontemporal_load(reinterpret_cast<const u16x4u *>(z + 2ll * at));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * j + i] = dev::lo16<KIND == COLI_PROB_BF16>(v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = -__builtin_inff();
                if (at + i < a.vocab) {
                    if constexpr (KIND == COLI_PROB_F32) v = *reinterpret_cast<const float *>(z + 4ll * (at + i));
                    else v = dev::lo16<KIND == COLI_PROB_BF16>(*reinterpret_cast<const uint16_t *>(z + 2ll * (at + i)));
                }
                x[4 * j + i] = v;
            }
        }
    }
    if (tid == 0) s_count = 0;
    float most = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        x[e] = fmaxf(x[e], -__builtin_inff());                        // NaN counts as -inf
        most = fmaxf(most, x[e]);
    }
    const uint32_t mine = key_of(most);
    float top = most;
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    float sum = 0.0f;
    if (fabsf(top) < 0x1p16f) {
        // 2^(z log2 e - top log2 e) by one multiply-add, rounded where it is small; the
        // rounding of the product with top, the same for all, is taken back behind the sum:
        // 2^-8 at most here, and a power of two near 1.  (It grows with top: from 2^31 on that
        // power can leave the range of fp32.)
        const float c = top * kLog2e, left = __builtin_fmaf(top, kLog2e, -c);
#pragma unroll
        for (int e = 0; e < EACH; ++e) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], kLog2e, -c));
        sum *= __builtin_amdgcn_exp2f(-left);
    } else if (top > -__builtin_inff()) {
#pragma unroll
        for (int e = 0; e < EACH; ++e) sum += __builtin_amdgcn_exp2f((x[e] - top) * kLog2e);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o, 64);
    const uint32_t reach = reached(mine, keep);
    if (lane == 0) {
        s_max[wave] = top;
        s_sum[wave] = sum;
        s_reach[wave] = reach;
    }
    __syncthreads();
    uint32_t limit = kLeastKey;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) limit = max(limit, s_reach[w]);
    const int group = row / a.beams, beam = row - group * a.beams;
    auto id_of = [&](int e) { return static_cast<uint32_t>(beam << kTokenBits | (first + ((e >> 2) * kThreads + tid) * 4 + (e & 3))); };
    const float least = value_of(limit);
    // The threshold is reached by few: a wave looks at one element of all lanes at a time,
    // first to count them, so that it takes its places of the list at once.
    int found = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) found += __popcll(__ballot(x[e] >= least));
    if (found) {
        int to = 0;
        if (lane == 0) to = atomicAdd(&s_count, found);
        to = __builtin_amdgcn_readfirstlane(to);
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const uint64_t m = __ballot(x[e] >= least);
            if (m) {
                const int at = to + __popcll(m & ((1ull << lane) - 1));
                if (x[e] >= least && at < kCandidates) s_cand[at] = packed(key_of(x[e]), id_of(e));
                to += __popcll(m);
            }
        }
    }
    __syncthreads();
    const int64_t part = static_cast<int64_t>(row) * chunks + chunk;
    if (tid == 0) {
        float m = s_max[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, s_max[w]);
        float l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            if (s_max[w] > -__builtin_inff()) l += s_sum[w] * __builtin_amdgcn_exp2f((s_max[w] - m) * kLog2e);
        a.sums[part] = float2{m, l};
    }
    // A group's lists lie place by place: the firsts of all lists, the seconds, ...
    const int lists = a.beams * chunks;
    uint64_t *best = a.best + static_cast<int64_t>(group) * lists * keep + beam * chunks + chunk;
    const int n = s_count;
    if (n <= kCandidates) {
        for (int i = tid; i < max(n, keep); i += kThreads) {
            if (i >= n) {
                best[i * lists] = 0;
                continue;
            }
            const uint64_t k = s_cand[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) rank += s_cand[j] > k;
            if (rank < keep) best[rank * lists] = k;
        }
        return;
    }
    // More at the threshold than are ranked (many equal logits, or keep near 64): one maximum
    // after the other.
    uint64_t before = ~0ull;
    for (int r = 0; r < keep; ++r) {
        uint64_t k = 0;
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const uint32_t key = key_of(x[e]);
            const uint64_t v = key ? packed(key, id_of(e)) : 0ull;
            if (v < before && v > k) k = v;
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const uint64_t other = __shfl_xor(k, o, 64);
            k = other > k ? other : k;
        }
        __syncthreads();
        if (lane == 0) s_top[wave] = k;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) k = s_top[w] > k ? s_top[w] : k;
        if (tid == 0) best[r * lists] = k;
        before = k;                                       // 0 once there is none left: v < 0 holds for nothing
    }
}

// A candidate's place: by score, then by beam, by logit (two of one beam may have scores
// that are the same in 64 bits; the greater logit is the first then as in the chunks' lists)
// and by token.  `rest` holds the three one above the other, the logit as its key's
// complement.  (No branches: of what is compared in a loop each would cost more than the rest.)
struct Candidate {
    double score;
    uint64_t rest;
    __device__ bool before(const Candidate &o) const { return (score > o.score) | ((score == o.score) & (rest < o.rest)); }
};

__global__ __launch_bounds__(kJoinThreads) void select_join_kernel(SelectArgs a, int group0, int chunks) {
    __shared__ Candidate s_cand[kJoinCandidates];
    __shared__ double s_add[kBeamMost];
    __shared__ float s_most[kBeamMost];
    __shared__ uint32_t s_reach[kJoinThreads / 64];
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 63, wave = dev::wave_id();
    const int g = blockIdx.x, keep = a.keep, w = a.beams;
    const int64_t out = (static_cast<int64_t>(group0) + g) * keep;
    if (tid == 0) s_count = 0;
    // The first candidates are asked for before anything else, all at once, and stay in registers.
    // They lie by their places in the chunks' lists, the first of every list before the second
    // of any: the lanes of the first waves then hold firsts alone, and the threshold is near.
    const int all = w * chunks * keep;
    const uint64_t *best = a.best + static_cast<int64_t>(g) * all;
    uint64_t held[kHeld];
#pragma unroll
    for (int r = 0; r < kHeld; ++r) held[r] = tid + r * kJoinThreads < all ? best[tid + r * kJoinThreads] : 0ull;
    // A row's greatest logit, which its logits are taken from first (in 64 bits a logit of
    // 1e20 would swallow the rest), and what is added then: its beam's score less the
    // logarithm of the sum.
    bool bad = false;
    for (int b = wave; b < w; b += kJoinThreads / 64) {
        const float2 *sums = a.sums + (static_cast<int64_t>(g) * w + b) * chunks;
        const float2 mine = lane < chunks ? sums[lane] : float2{-__builtin_inff(), 0.0f};
        const float score = a.scores[(static_cast<int64_t>(group0) + g) * w + b];
        float m = mine.x;
        for (int i = lane + 64; i < chunks; i += 64) m = fmaxf(m, sums[i].x);
#pragma unroll
        for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
        auto part = [&](const float2 &v) { return v.x > -__builtin_inff() ? static_cast<double>(v.y) * __builtin_amdgcn_exp2f((v.x - m) * kLog2e) : 0.0; };
        double l = part(mine);
        for (int i = lane + 64; i < chunks; i += 64) l += part(sums[i]);
#pragma unroll
        for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o, 64);
        const bool live = __builtin_isfinite(score), some = __builtin_isfinite(m);
        if (lane == 0) {
            s_most[b] = m;
            s_add[b] = live && some ? static_cast<double>(score) - log(l) : -__builtin_inf();
        }
        bad = bad || (live && !some);
    }
    dev::flag_if(bad && lane == 0, a.err, kErrNoMass);
    __syncthreads();
    auto read = [&](uint64_t k, Candidate &c) {
        if (k == 0) return false;
        const uint32_t id = ~static_cast<uint32_t>(k), key = static_cast<uint32_t>(k >> 32);
        const int b = id >> kTokenBits;
        c.rest = static_cast<uint64_t>(b) << (32 + kTokenBits) | static_cast<uint64_t>(~key) << kTokenBits | (id & ((1u << kTokenBits) - 1));
        c.score = s_add[b] + (static_cast<double>(value_of(key)) - s_most[b]);
        return c.score > -__builtin_inf();
    };
    auto each = [&](auto f) {
#pragma unroll
        for (int r = 0; r < kHeld; ++r) {
            Candidate c;
            if (read(held[r], c)) f(c);
        }
        for (int i = tid + kHeld * kJoinThreads; i < all; i += kJoinThreads) {
            Candidate c;
            if (read(best[i], c)) f(c);
        }
    };
    // The threshold as in a chunk, on the scores rounded to 32 bits: rounding keeps
    // the order, so that what is below it is behind the candidates that reach it.  (A
    // score below the range of 32 bits has the smallest key that a candidate has.)
    auto key = [&](const Candidate &c) { return max(key_of(static_cast<float>(c.score)), kLeastKey); };
    uint32_t mine = 0;
    each([&](const Candidate &c) { mine = max(mine, key(c)); });
    const uint32_t reach = reached(mine, keep);
    if (lane == 0) s_reach[wave] = reach;
    __syncthreads();
    uint32_t limit = kLeastKey;
#pragma unroll
    for (int v = 0; v < kJoinThreads / 64; ++v) limit = max(limit, s_reach[v]);
    if (mine >= limit)
        each([&](const Candidate &c) {
            if (key(c) < limit) return;
            const int at = atomicAdd(&s_count, 1);
            if (at < kJoinCandidates) s_cand[at] = c;
        });
    __syncthreads();
    auto put = [&](int r, const Candidate &c) {
        a.out_scores[out + r] = static_cast<float>(c.score);
        a.parents[out + r] = static_cast<int32_t>(c.rest >> (32 + kTokenBits));
        a.tokens[out + r] = static_cast<int32_t>(c.rest & ((1u << kTokenBits) - 1));
    };
    auto put_none = [&](int r) {
        a.out_scores[out + r] = -__builtin_inff();
        a.parents[out + r] = -1;
        a.tokens[out + r] = -1;
    };
    const int n = s_count;
    if (n <= kJoinCandidates) {
        for (int i = tid; i < max(n, keep); i += kJoinThreads) {
            if (i >= n) {
                put_none(i);
                continue;
            }
            const Candidate mine = s_cand[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) rank += s_cand[j].before(mine);
            if (rank < keep) put(rank, mine);
        }
        return;
    }
    // Many equal scores: one after the other.
    __shared__ Candidate s_top[kJoinThreads / 64];
    __shared__ Candidate s_last;
    for (int r = 0; r < keep; ++r) {
        Candidate k{-__builtin_inf(), ~0ull};
        each([&](const Candidate &c) {
            if ((r == 0 || s_last.before(c)) && c.before(k)) k = c;
        });
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const Candidate other{__shfl_xor(k.score, o, 64), __shfl_xor(k.rest, o, 64)};
            if (other.before(k)) k = other;
        }
        if (lane == 0) s_top[wave] = k;
        __syncthreads();
        if (tid == 0) {
            for (int v = 1; v < kJoinThreads / 64; ++v)
                if (s_top[v].before(k)) k = s_top[v];
            s_last = k;
            put(r, k);                                    // there are more of them than `keep`
        }
        __syncthreads();
    }
}

template <int EACH>
void launch_chunks(const SelectArgs &a, int row0, int rows, int chunks, hipStream_t s) {
    launch(a.kind == COLI_PROB_F32    ? select_kernel<COLI_PROB_F32, EACH>
           : a.kind == COLI_PROB_BF16 ? select_kernel<COLI_PROB_BF16, EACH>
                                      : select_kernel<COLI_PROB_F16, EACH>,
           static_cast<unsigned>(rows) * chunks, kThreads, 0, s, a, row0, chunks);
}

}  // namespace

hipError_t launch_select(const SelectArgs &a, int n_cu, hipStream_t s) {
    // Chunks of 8192 elements; of 2048 where those are few: replayed from a graph, 4 rows of
    // 32000 take 9.1 us in small and 10.6 in large ones, one of 151643 9.3 and 10.5, 4 of 151643
    // (76 large chunks) 11.1 and 11.0, 16 13.4 and 12.4, 256 69.6 and 42.4.  (4096 there: 49.)
    const int64_t rows = static_cast<int64_t>(a.n_groups) * a.beams;
    const bool small = rows * ((a.vocab + 8191) / 8192) < n_cu / 4;
    const int each = small ? 2048 : 8192, chunks = (a.vocab + each - 1) / each;
    // As many groups in a launch as the scratch holds.
    const int64_t per = static_cast<int64_t>(a.beams) * chunks;
    const int64_t most = std::min({a.best_cap / (per * a.keep), a.sums_cap / per, static_cast<int64_t>(INT32_MAX) / per});
    if (most < 1) return hipErrorInvalidValue;
    for (int64_t g = 0; g < a.n_groups; g += most) {
        const int n = static_cast<int>(std::min<int64_t>(most, a.n_groups - g));
        if (small) launch_chunks<8>(a, static_cast<int>(g) * a.beams, n * a.beams, chunks, s);
        else launch_chunks<32>(a, static_cast<int>(g) * a.beams, n * a.beams, chunks, s);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        launch(select_join_kernel, static_cast<unsigned>(n), kJoinThreads, 0, s, a, static_cast<int>(g), chunks);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace coli
