// verify.hip -- acceptance of drafted tokens against the target's
// probabilities, for chains and trees, from given random numbers.
//
// At a node with target row p and (optional) draft row q the children are
// tried in node order.  After k refusals the residual is r_k = (p - a_k q)+ /
// Z_k with a_0 = 0, Z_0 = 1, a_{k+1} = a_k + Z_k and Z_k = sum (p - a_k q)+
// (subtracting q from a normalised residual and normalising again only moves
// a), and child x is taken when u q(x) Z_k < (p - a_k q)+(x).  Without draft
// rows a child's q is the point mass of its token: r_k is p without the
// refused tokens and Z_k = 1 - their probability.  Where no child is taken the
// next token is the one of the largest r race, race = 1 / Exp(1): that draws
// from r, needs no sum over the row, and is the same for every split of it.
//
// One launch: a sequence's workgroups each make the walk (a few gathers,
// loaded together) and take a slice of the final row; the slices meet in a
// 64-bit maximum of (score, lowest index).  Trees with draft rows need the sums
// Z_k of the nodes they stop at, so their walk is a launch of its own, one
// workgroup per sequence.  The floor is the final row of p, q and race.
#include "coli_moe.h"
#include "dev_attn.h"

namespace coli {
namespace {

constexpr int kSampleThreads = 256, kWalkThreads = 1024;
// A workgroup takes its slice of a row in chunks of four groups of four elements
// per thread, all in flight at once; the first of race is loaded before the
// walk, which says which row of p it meets.  Slices are one to four chunks,
// as many as let every workgroup (five fit a CU) start at once: each makes the
// walk again.  64 sequences of 151643 fp32 probabilities, 78 MB: two chunks 22 us,
// 3.5 TB/s, of which the walk takes 3.6 us; one chunk (two rounds of
// workgroups) 31.5 us; 16384 elements in 16 rounds of one group 24.3 us.
constexpr int kGroups = 4;
constexpr int kChunk = kSampleThreads * 4 * kGroups;
constexpr int kMostChunks = 4;
constexpr int kPerCU = 5;

enum Kind { kF32 = COLI_PROB_F32, kBF16 = COLI_PROB_BF16, kF16 = COLI_PROB_F16 };

template <int K>
__device__ __forceinline__ float prob(const uint8_t *row, int i) {
    if constexpr (K == kF32) return *reinterpret_cast<const float *>(row + 4ll * i);
    const uint32_t w = *reinterpret_cast<const uint16_t *>(row + 2ll * i);
    return dev::lo16<K == kBF16>(w);
}
// Four values from element i on.  Rows need only their element's alignment
// (a row of an odd vocabulary starts anywhere).
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));
template <int K>
__device__ __forceinline__ void prob4(const uint8_t *row, int i, float (&v)[4]) {
    if constexpr (K == kF32) {
        const f32x4u x = *reinterpret_cast<const f32x4u *>(row + 4ll * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = x[j];
    } else {
        const u16x4u x = *reinterpret_cast<const u16x4u *>(row + 2ll * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = dev::lo16<K == kBF16>(x[j]);
    }
}
template <int K>
constexpr int prob_bytes() { return K == kF32 ? 4 : 2; }

// Negative and NaN probabilities count as zero.
__device__ __forceinline__ float counted(float v) { return v > 0.0f ? v : 0.0f; }

// (p - a q)+, each operation rounded on its own (no fused multiply-add).  (A p
// of no value leaves nothing as it stands.)
__device__ __forceinline__ float residual(float p, float a, float q) {
#pragma clang fp contract(off)
    const float t = a * counted(q);
    const float r = p - t;
    return r > 0.0f ? r : 0.0f;
}

struct Walk {
    int node;       // where the walk ended
    int refused;    // its children, all refused
    float over;     // a of the residual that the next token is drawn from
};

// The nodes of one sequence: what each node's test needs, loaded at once.
struct Nodes {
    float p[kVerifyMaxNodes], q[kVerifyMaxNodes], u[kVerifyMaxNodes];
    int x[kVerifyMaxNodes], parent[kVerifyMaxNodes];
    int path[kVerifyMaxNodes];
    float sum[kWalkThreads / 64];
    int n, steps, cur, refused, again;
    float over, left;
};

// Walks from node 0.  Every thread of the workgroup calls it; SUMS also
// computes Z_k where a second child is tried (only then do threads beside
// the first wave take part).
template <int K, int NT, bool SUMS>
__device__ __forceinline__ Walk walk(const VerifyArgs &a, int t0, int n, Nodes &s, bool &bad) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int j = tid; j < n; j += NT) {
        int parent = a.parents ? a.parents[t0 + j] : j - 1;
        const int x = a.tokens[t0 + j];
        bool ok = j > 0;
        if (ok && (parent < 0 || parent >= j || x < 0 || x >= a.vocab)) {
            bad = true;
            ok = false;
        }
        float p = 0.0f, q = 1.0f;
        if (ok) {
            p = counted(prob<K>(a.p + (t0 + parent) * a.p_stride * prob_bytes<K>(), x));
            if (a.q) q = counted(prob<K>(a.q + (t0 + parent) * a.q_stride * prob_bytes<K>(), x));
        } else {
            parent = -1;
        }
        s.p[j] = p;
        s.q[j] = q;
        s.u[j] = a.u[t0 + j];
        s.x[j] = x;
        s.parent[j] = parent;
    }
    if (tid == 0) {
        s.steps = 1;
        s.path[0] = 0;
        s.cur = 0;
        s.refused = 0;
        s.over = 0.0f;
        s.left = 1.0f;
        s.again = 1;
    }
    __syncthreads();
    // The first wave walks; with SUMS it stops (again = 2) where a residual's
    // sum is needed.  `from` is the first node not yet tried as a child.
    int from = 1;
    while (true) {
        if (wave == 0) {
            int cur = s.cur, refused = s.refused, steps = s.steps, state = 0;
            float over = s.over, left = s.left;
            bool stale = false;                          // left is not yet the sum at over
            const int cap = min(a.path_cols, n);
            while (state == 0) {
                int child = -1;
                for (int b = from & ~63; b < n; b += 64) {
                    const int j = b + lane;
                    const uint64_t hit = __ballot(j >= from && j < n && s.parent[j] == cur);
                    if (hit) {
                        child = b + __ffsll(static_cast<unsigned long long>(hit)) - 1;
                        break;
                    }
                }
                if (child < 0 || steps >= cap) {
                    state = 1;
                    break;
                }
                if (SUMS && stale) {
                    from = child;
                    state = 2;
                    break;
                }
                from = child + 1;
                float px = s.p[child];
                bool take;
                if (a.q) {
                    take = s.u[child] * s.q[child] * left < residual(px, over, s.q[child]);
                } else {
                    // A token that was refused has no probability left.
                    for (int b = (cur + 1) & ~63; b < child; b += 64) {
                        const int j = b + lane;
                        if (__any(j > cur && j < child && s.parent[j] == cur && s.x[j] == s.x[child])) px = 0.0f;
                    }
                    take = s.u[child] * left < px;
                }
                if (take) {
                    cur = child;
                    if (lane == 0) s.path[steps] = child;
                    ++steps;
                    refused = 0;
                    over = 0.0f;
                    left = 1.0f;
                } else {
                    ++refused;
                    if (a.q) {
                        over = over + left;
                        stale = true;
                    } else {
                        left = left - px;
                    }
                }
            }
            if (lane == 0) {
                s.cur = cur;
                s.refused = refused;
                s.steps = steps;
                s.over = over;
                s.left = left;
                s.again = state;
            }
        }
        __syncthreads();
        if (!SUMS || s.again != 2) break;
        // Z of the residual at s.over: the whole row, in a fixed order.
        const uint8_t *p = a.p + (t0 + s.cur) * a.p_stride * prob_bytes<K>();
        const uint8_t *q = a.q + (t0 + s.cur) * a.q_stride * prob_bytes<K>();
        const float over = s.over;
        float sum = 0.0f;
        int i = 4 * tid;
        for (; i + 4 <= a.vocab; i += 4 * NT) {
            float pv[4], qv[4];
            prob4<K>(p, i, pv);
            prob4<K>(q, i, qv);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += residual(pv[j], over, qv[j]);
        }
        for (; i < a.vocab; ++i) sum += residual(prob<K>(p, i), over, prob<K>(q, i));
#pragma unroll
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o, 64);
        if (lane == 0) s.sum[wave] = sum;
        __syncthreads();
        if (tid == 0) {
            float z = 0.0f;
            for (int w = 0; w < NT / 64; ++w) z += s.sum[w];
            s.left = z;
        }
        __syncthreads();
    }
    return Walk{s.cur, s.refused, s.over};
}

// The path, its length and the accepted tokens of one sequence; the sampled
// token follows them.
__device__ __forceinline__ void write_path(const VerifyArgs &a, int seq, const Nodes &s, int n, int nt) {
    const int64_t at = static_cast<int64_t>(seq) * a.path_cols;
    for (int i = threadIdx.x; i < a.path_cols; i += nt) {
        a.path[at + i] = n > 0 && i < s.steps ? s.path[i] : -1;
        if (n <= 0 || i != s.steps - 1) a.out_tokens[at + i] = n > 0 && i + 1 < s.steps ? s.x[s.path[i + 1]] : -1;
    }
    if (threadIdx.x == 0) a.count[seq] = n > 0 ? s.steps : 0;
}

// The sequence's first token and node count; false (and 0 nodes) where its
// bounds are outside the call.
__device__ __forceinline__ bool bounds(const VerifyArgs &a, int seq, int &t0, int &n) {
    t0 = a.q_start[seq];
    const int t1 = a.q_start[seq + 1];
    n = t1 - t0;
    const bool ok = t0 >= 0 && n >= 0 && t1 <= a.n_tok;
    if (!ok) n = 0;
    n = min(n, kVerifyMaxNodes);
    return ok && t1 - t0 <= kVerifyMaxNodes;
}

template <int K>
__global__ __launch_bounds__(kWalkThreads) void walk_kernel(VerifyArgs a) {
    __shared__ Nodes s;
    const int seq = blockIdx.x;
    int t0, n;
    bool bad = false;
    dev::flag_if(!bounds(a, seq, t0, n) && threadIdx.x == 0, a.err, kErrSeq);
    Walk w{0, 0, 0.0f};
    if (n > 0) w = walk<K, kWalkThreads, true>(a, t0, n, s, bad);
    dev::flag_if(bad, a.err, kErrDraft);
    write_path(a, seq, s, n, kWalkThreads);
    if (threadIdx.x == 0) {
        int32_t *o = a.walk + 4 * seq;
        o[0] = w.node;
        o[1] = w.refused;
        o[2] = __float_as_int(w.over);
        o[3] = n > 0 ? s.steps : 0;
    }
}

// Orders candidates by score, then by lowest index; zero is no candidate.
__device__ __forceinline__ uint64_t candidate(float score, int i) {
    return score >= 0.0f ? (static_cast<uint64_t>(__float_as_uint(score + 0.0f) + 1u) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i)) : 0ull;
}

template <int K, bool WALKED>
__global__ __launch_bounds__(kSampleThreads, kPerCU) void sample_kernel(VerifyArgs a, int chunks) {
    __shared__ Nodes s;
    __shared__ uint32_t s_gone[kMostChunks * kChunk / 32];   // bits of the refused tokens
    __shared__ uint64_t s_best[2][kSampleThreads / 64];
    const int seq = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool first = blockIdx.x == 0;
    const int lo = blockIdx.x * chunks * kChunk, hi = min(lo + chunks * kChunk, a.vocab);
    const float *race = a.race + seq * a.race_stride;
    f32x4u g[kGroups];
    auto load_race = [&](int c, f32x4u (&to)[kGroups]) {
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int i = lo + c * kChunk + 4 * (tid + k * kSampleThreads);
            to[k] = f32x4u{0.0f, 0.0f, 0.0f, 0.0f};
            if (i + 4 <= hi) to[k] = *reinterpret_cast<const f32x4u *>(race + i);
        }
    };
    load_race(0, g);
    int t0, n, steps;
    bool bad = false;
    const bool ok = bounds(a, seq, t0, n);
    Walk w;
    if constexpr (WALKED) {
        const int32_t *o = a.walk + 4 * seq;
        w = Walk{o[0], o[1], __int_as_float(o[2])};
        steps = o[3];
        if (n <= 0) return;
    } else {
        dev::flag_if(!ok && first && tid == 0, a.err, kErrSeq);
        if (n <= 0) {
            if (first) write_path(a, seq, s, n, kSampleThreads);
            return;
        }
        w = walk<K, kSampleThreads, false>(a, t0, n, s, bad);
        if (first) {
            dev::flag_if(bad, a.err, kErrDraft);
            write_path(a, seq, s, n, kSampleThreads);
        }
        steps = s.steps;
    }
    const bool remove = !WALKED && !a.q && w.refused > 0;   // refused tokens without draft rows
    if (remove) {
        for (int i = tid; i < kMostChunks * kChunk / 32; i += kSampleThreads) s_gone[i] = 0;
        __syncthreads();
        for (int j = w.node + 1 + tid; j < n; j += kSampleThreads)
            if (s.parent[j] == w.node && s.x[j] >= lo && s.x[j] < hi)
                atomicOr(&s_gone[(s.x[j] - lo) >> 5], 1u << ((s.x[j] - lo) & 31));
        __syncthreads();
    }
    const uint8_t *p = a.p + (t0 + w.node) * a.p_stride * prob_bytes<K>();
    const uint8_t *q = a.q ? a.q + (t0 + w.node) * a.q_stride * prob_bytes<K>() : nullptr;
    const bool drawn = q && w.refused > 0;
    // The best of the residual, and of p itself where the residual is nothing.
    uint64_t best = 0, whole = 0;
    auto one = [&](int i, float pv, float qv, float g, bool gone) {
        if (!(pv > 0.0f)) return;
        const float left = drawn ? residual(pv, w.over, qv) : gone ? 0.0f : pv;
        if (left > 0.0f) {
            const uint64_t c = candidate(left * g, i);
            best = c > best ? c : best;
        }
        const uint64_t c = candidate(pv * g, i);
        whole = c > whole ? c : whole;
    };
    for (int c = 0; c < chunks; ++c) {
        const int at = lo + c * kChunk;
        float pv[kGroups][4], qv[kGroups][4];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int i = at + 4 * (tid + k * kSampleThreads);
#pragma unroll
            for (int j = 0; j < 4; ++j) pv[k][j] = qv[k][j] = 0.0f;
            if (i + 4 <= hi) {
                prob4<K>(p, i, pv[k]);
                if (drawn) prob4<K>(q, i, qv[k]);
            }
        }
        if (c > 0) load_race(c, g);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int i = at + 4 * (tid + k * kSampleThreads);
            if (i >= hi) continue;
            const uint32_t gone = remove ? s_gone[(i - lo) >> 5] >> ((i - lo) & 31) : 0u;
            if (i + 4 <= hi) {
#pragma unroll
                for (int j = 0; j < 4; ++j) one(i + j, pv[k][j], qv[k][j], g[k][j], (gone >> j) & 1);
            } else {
                for (int j = 0; i + j < hi; ++j)
                    one(i + j, prob<K>(p, i + j), drawn ? prob<K>(q, i + j) : 0.0f, race[i + j], (gone >> j) & 1);
            }
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const uint64_t x = __shfl_xor(static_cast<unsigned long long>(best), o, 64);
        const uint64_t y = __shfl_xor(static_cast<unsigned long long>(whole), o, 64);
        best = x > best ? x : best;
        whole = y > whole ? y : whole;
    }
    if (lane == 0) {
        s_best[0][wave] = best;
        s_best[1][wave] = whole;
    }
    __syncthreads();
    unsigned long long *out = reinterpret_cast<unsigned long long *>(a.best) + 2 * seq;
    if (tid < 2) {
        uint64_t v = 0;
        for (int k = 0; k < kSampleThreads / 64; ++k) v = s_best[tid][k] > v ? s_best[tid][k] : v;
        if (v) __hip_atomic_fetch_max(out + tid, static_cast<unsigned long long>(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!dev::arrive_last(a.arrived + seq, static_cast<int>(gridDim.x))) return;
    if (tid == 0) {
        uint64_t v = __hip_atomic_exchange(out, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint64_t rest = __hip_atomic_exchange(out + 1, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (!v) v = rest;
        const int token = v ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(v)) : 0;
        dev::flag_if(!v, a.err, kErrNoMass);
        a.out_tokens[static_cast<int64_t>(seq) * a.path_cols + steps - 1] = token;
    }
}

template <int K>
hipError_t launch_kind(const VerifyArgs &a, int n_cu, hipStream_t s) {
    const int64_t want = (static_cast<int64_t>(a.vocab) * a.n_seq + static_cast<int64_t>(kPerCU) * n_cu * kChunk - 1) / (static_cast<int64_t>(kPerCU) * n_cu * kChunk);
    const int chunks = static_cast<int>(std::min<int64_t>(std::max<int64_t>(want, 1), kMostChunks));
    const unsigned slices = static_cast<unsigned>((a.vocab + chunks * kChunk - 1) / (chunks * kChunk));
    // A call without nodes has only paths of nothing to write: its probabilities
    // and race may be NULL, and sampling loads race before it knows of any node.
    const bool sums = a.q && a.parents;
    if (sums || a.n_tok == 0) {
        launch(walk_kernel<K>, static_cast<unsigned>(a.n_seq), kWalkThreads, 0, s, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || a.n_tok == 0) return e;
        launch(sample_kernel<K, true>, dim3(slices, a.n_seq), kSampleThreads, 0, s, a, chunks);
    } else {
        launch(sample_kernel<K, false>, dim3(slices, a.n_seq), kSampleThreads, 0, s, a, chunks);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, int n_cu, hipStream_t s) {
    switch (a.kind) {
        case kF32: return launch_kind<kF32>(a, n_cu, s);
        case kBF16: return launch_kind<kBF16>(a, n_cu, s);
        default: return launch_kind<kF16>(a, n_cu, s);
    }
}

}  // namespace coli
