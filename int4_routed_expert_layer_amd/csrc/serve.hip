// serve.hip -- host side of the serving operators declared in
// include/coli_moe.h: the handle with its plan and scratch, argument checks,
// launches.
#include <cstdarg>
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>
#include <string>

#include "coli_moe.h"
#include "serve.h"

using namespace coli;

struct coli_serve {
    coli_serve_dims d{};
    int device = 0;
    int n_cu = 0;
    DecodePlan plan{};
    float *part = nullptr;
    float *part_ml = nullptr;
    int32_t *walk = nullptr;
    uint64_t *best = nullptr;
    int32_t *arrived = nullptr;
    int32_t *err = nullptr;
    int plan_tok = -1, plan_seq = 0;   // sizes of the current plan, -1: none yet
    std::string msg;
};

namespace {

thread_local std::string g_serve_error;

coli_status fail(coli_serve *S, coli_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    try {
        (S ? S->msg : g_serve_error) = buf;
    } catch (...) {   // no memory for the text: the code alone
    }
    return st;
}

coli_status launched(coli_serve *S, hipError_t e, const char *what) {
    if (e == hipSuccess) return COLI_OK;
    return fail(S, COLI_E_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

struct OnDevice {
    int prev = -1;
    bool ok = false;
    explicit OnDevice(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) prev = -1;
        ok = prev == dev || hipSetDevice(dev) == hipSuccess;
        if (prev == dev) prev = -1;
    }
    ~OnDevice() {
        if (prev >= 0) (void)hipSetDevice(prev);
    }
};

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Floats of statistics per row of a slot: two for absorbed attention, up to eight for
// expanded, whose parts have fewer outputs.
constexpr int kSlotStats = 8;

struct Sizes {
    int64_t items, joins, slots, seqs;
};
// Room of a plan: one item per 64-row unit (each sequence may end in a part of
// one), and four rounds over the CUs of pieces; pieces of cut units hold
// partial results.
Sizes plan_sizes(const coli_serve_dims &d, int n_cu) {
    const int64_t units = static_cast<int64_t>(d.max_tokens) * d.n_heads / kTileRows + d.max_seqs;
    const int64_t slots = 4ll * n_cu;
    const int64_t rounds = (units + slots + n_cu - 1) / n_cu + 1;
    return Sizes{rounds * n_cu, std::min(units, slots / 2), slots, d.max_seqs};
}
size_t create_bytes(const coli_serve_dims &d, int n_cu) {
    const Sizes z = plan_sizes(d, n_cu);
    return static_cast<size_t>(z.items) * sizeof(DecodeItem) + static_cast<size_t>(z.joins) * sizeof(JoinUnit) +
           static_cast<size_t>(z.slots) * kTileRows * (kLatent + kSlotStats) * sizeof(float) +
           static_cast<size_t>(z.seqs) * (8 * sizeof(int32_t) + 2 * sizeof(uint64_t) + sizeof(int32_t)) + 5 * sizeof(int32_t);
}

void free_serve(coli_serve *S) {
    void *ptrs[] = {S->plan.head, S->plan.items, S->plan.joins, S->plan.seq, S->part, S->part_ml, S->walk, S->best, S->arrived, S->err};
    for (void *p : ptrs) book_free(p);
    delete S;
}

// The cache arguments shared by the calls that use it.
coli_status check_cache(coli_serve *S, const void *cache, int64_t page_stride, int32_t n_pages) {
    if (!cache) return fail(S, COLI_E_INVALID, "cache is NULL");
    if (!aligned(cache, 16)) return fail(S, COLI_E_INVALID, "cache must be 16-byte aligned");
    if (n_pages < 1) return fail(S, COLI_E_INVALID, "n_pages %d must be >= 1", n_pages);
    const int64_t page = static_cast<int64_t>(S->d.page_size) * kCacheRow;
    if (page_stride < page || page_stride % 8)
        return fail(S, COLI_E_INVALID, "page_stride %lld must be a multiple of 8 and >= page_size * %d = %lld",
                    static_cast<long long>(page_stride), kCacheRow, static_cast<long long>(page));
    return COLI_OK;
}

CacheView view(const coli_serve *S, const void *cache, int64_t page_stride, int32_t n_pages, const int32_t *table,
               int64_t table_stride, int32_t table_cols) {
    CacheView v{};
    v.base = static_cast<uint8_t *>(const_cast<void *>(cache));
    v.page_stride = page_stride;
    v.n_pages = n_pages;
    v.page_shift = __builtin_ctz(static_cast<unsigned>(S->d.page_size));
    // A table without columns: some address that can be read; every page is out of range.
    v.table = table_cols > 0 ? table : S->err;
    v.table_stride = table_cols > 0 ? table_stride : 0;
    v.table_cols = table_cols;
    return v;
}

coli_status check_counts(coli_serve *S, int32_t n_tok, int32_t n_seq) {
    if (n_tok < 0 || n_tok > S->d.max_tokens) return fail(S, COLI_E_INVALID, "n_tok %d must be in 0..max_tokens (%d)", n_tok, S->d.max_tokens);
    if (n_seq < 0 || n_seq > S->d.max_seqs) return fail(S, COLI_E_INVALID, "n_seq %d must be in 0..max_seqs (%d)", n_seq, S->d.max_seqs);
    return COLI_OK;
}

#define CHECK(call)                                   \
    do {                                              \
        const coli_status st_ = (call);               \
        if (st_ != COLI_OK) return st_;               \
    } while (0)
#define NEED(cond, ...)                                                \
    do {                                                               \
        if (!(cond)) return fail(S, COLI_E_INVALID, __VA_ARGS__);      \
    } while (0)

}  // namespace

extern "C" {

coli_status coli_serve_create(const coli_serve_dims *d, int device, coli_serve **out) {
    coli_serve *S = nullptr;
    NEED(out, "out is NULL");
    NEED(d, "dims is NULL");
    NEED(d->n_heads > 0 && d->max_tokens > 0 && d->max_seqs > 0, "n_heads, max_tokens and max_seqs must be positive");
    NEED(d->page_size > 0 && (d->page_size & (d->page_size - 1)) == 0 && d->page_size <= 65536, "page_size %d must be a power of two up to 65536", d->page_size);
    NEED(d->half == COLI_HALF_BF16 || d->half == COLI_HALF_F16, "half must be COLI_HALF_BF16 or COLI_HALF_F16");
    if (d->latent != kLatent || d->rope != kRope)
        return fail(nullptr, COLI_E_UNSUPPORTED, "latent %d and rope %d: %d and %d are supported", d->latent, d->rope, kLatent, kRope);
    if (!((d->nope == 192 && d->v_dim == 256) || (d->nope == 128 && d->v_dim == 128)))
        return fail(nullptr, COLI_E_UNSUPPORTED, "nope %d with v_dim %d: 192 with 256 and 128 with 128 are supported", d->nope, d->v_dim);
    if (d->n_heads > 1024 || static_cast<int64_t>(d->max_tokens) * d->n_heads > (1 << 30) || d->max_seqs > (1 << 20))
        return fail(nullptr, COLI_E_UNSUPPORTED, "n_heads must be <= 1024, max_tokens * n_heads <= 2^30 and max_seqs <= 2^20");
    if (!book_fits(create_bytes(*d, 256))) return fail(nullptr, COLI_E_NOMEM, "allocation cap: the handle needs %zu bytes", create_bytes(*d, 256));
    int ndev = 0;
    hipError_t he = hipGetDeviceCount(&ndev);
    if (he != hipSuccess || ndev <= 0) return fail(nullptr, COLI_E_DEVICE, "no HIP device available (%s)", hipGetErrorString(he));
    NEED(device >= 0 && device < ndev, "device %d out of range", device);
    OnDevice on(device);
    if (!on.ok) return fail(nullptr, COLI_E_DEVICE, "cannot select device %d", device);
    int n_cu = 0;
    if ((he = hipDeviceGetAttribute(&n_cu, hipDeviceAttributeMultiprocessorCount, device)) != hipSuccess)
        return fail(nullptr, COLI_E_DEVICE, "hipDeviceGetAttribute: %s", hipGetErrorString(he));
    S = new (std::nothrow) coli_serve();
    if (!S) return fail(nullptr, COLI_E_NOMEM, "no host memory for the handle");
    S->d = *d;
    S->device = device;
    S->n_cu = std::max(8, n_cu / 8 * 8);   // workgroups of a round: the same number on each of eight XCDs
    n_cu = S->n_cu;
    const Sizes z = plan_sizes(*d, n_cu);
    S->plan.item_cap = static_cast<int>(z.items);
    S->plan.join_cap = static_cast<int>(z.joins);
    S->plan.slot_cap = static_cast<int>(z.slots);
    struct { void **p; size_t n; const char *what; } allocs[] = {
        {reinterpret_cast<void **>(&S->plan.head), 4 * sizeof(int32_t), "plan head"},
        {reinterpret_cast<void **>(&S->plan.items), z.items * sizeof(DecodeItem), "plan items"},
        {reinterpret_cast<void **>(&S->plan.joins), z.joins * sizeof(JoinUnit), "plan joins"},
        {reinterpret_cast<void **>(&S->plan.seq), z.seqs * 4 * sizeof(int32_t), "plan scratch"},
        {reinterpret_cast<void **>(&S->part), z.slots * kTileRows * kLatent * sizeof(float), "partial outputs"},
        {reinterpret_cast<void **>(&S->part_ml), z.slots * kTileRows * kSlotStats * sizeof(float), "partial statistics"},
        {reinterpret_cast<void **>(&S->walk), z.seqs * 4 * sizeof(int32_t), "draft walks"},
        {reinterpret_cast<void **>(&S->best), z.seqs * 2 * sizeof(uint64_t), "sample maxima"},
        {reinterpret_cast<void **>(&S->arrived), z.seqs * sizeof(int32_t), "arrival counters"},
        {reinterpret_cast<void **>(&S->err), sizeof(int32_t), "error flags"},
    };
    for (auto &a : allocs)
        if ((he = book_alloc(a.p, a.n)) != hipSuccess) {
            const coli_status st = he == hipErrorOutOfMemory ? COLI_E_NOMEM : COLI_E_DEVICE;
            fail(nullptr, st, "hipMalloc %s (%zu bytes): %s", a.what, a.n, hipGetErrorString(he));
            free_serve(S);
            return st;
        }
    if ((he = hipMemset(S->best, 0, z.seqs * 2 * sizeof(uint64_t))) != hipSuccess ||
        (he = hipMemset(S->arrived, 0, z.seqs * sizeof(int32_t))) != hipSuccess ||
        (he = hipMemset(S->plan.head, 0, 4 * sizeof(int32_t))) != hipSuccess ||
        (he = hipMemset(S->plan.items, 0, z.items * sizeof(DecodeItem))) != hipSuccess ||
        (he = hipMemset(S->err, 0, sizeof(int32_t))) != hipSuccess || (he = hipDeviceSynchronize()) != hipSuccess) {
        fail(nullptr, COLI_E_DEVICE, "handle setup: %s", hipGetErrorString(he));
        free_serve(S);
        return COLI_E_DEVICE;
    }
    *out = S;
    return COLI_OK;
}

coli_status coli_serve_destroy(coli_serve *S) {
    if (!S) return COLI_OK;
    OnDevice on(S->device);
    (void)hipDeviceSynchronize();
    free_serve(S);
    return COLI_OK;
}

const char *coli_serve_last_error(const coli_serve *S) { return S ? S->msg.c_str() : g_serve_error.c_str(); }

coli_status coli_serve_device_errors(coli_serve *S, int32_t *flags) {
    NEED(S, "handle is NULL");
    NEED(flags, "flags is NULL");
    OnDevice on(S->device);
    hipError_t e = hipDeviceSynchronize();
    if (e == hipSuccess) e = hipMemcpy(flags, S->err, sizeof(int32_t), hipMemcpyDeviceToHost);
    if (e == hipSuccess) e = hipMemset(S->err, 0, sizeof(int32_t));
    if (e == hipSuccess) e = hipDeviceSynchronize();
    return launched(S, e, "error flags");
}

coli_status coli_latent_append(coli_serve *S, const void *c, int64_t c_stride, const void *norm_weight, float eps, const float *cos_table,
                               const float *sin_table, int32_t n_positions, int32_t interleaved, const int32_t *positions,
                               const int64_t *slots, int32_t n_tok, void *cache, int64_t page_stride, int32_t n_pages, const void *q_pe,
                               int64_t q_tok_stride, int64_t q_head_stride, void *q_out, void *stream) {
    NEED(S, "handle is NULL");
    CHECK(check_counts(S, n_tok, 0));
    CHECK(check_cache(S, cache, page_stride, n_pages));
    NEED(interleaved == 0 || interleaved == 1, "interleaved must be 0 or 1");
    NEED(n_positions >= 1, "n_positions %d must be >= 1", n_positions);
    NEED(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and >= 0");
    if (n_tok == 0) return COLI_OK;
    NEED(c && norm_weight && cos_table && sin_table && positions && slots, "NULL device pointer");
    NEED((q_pe == nullptr) == (q_out == nullptr), "q_pe and q_out go together");
    NEED(aligned(c, 16) && aligned(norm_weight, 16) && aligned(q_pe, 16) && aligned(q_out, 16), "c, norm_weight, q_pe and q_out must be 16-byte aligned");
    NEED(c_stride % 8 == 0 && q_tok_stride % 8 == 0 && q_head_stride % 8 == 0, "strides must be multiples of 8 elements");
    AppendArgs a{};
    a.c = static_cast<const uint8_t *>(c);
    a.weight = static_cast<const uint8_t *>(norm_weight);
    a.c_stride = c_stride;
    a.eps = eps;
    a.cos_t = cos_table;
    a.sin_t = sin_table;
    a.n_pos = n_positions;
    a.interleaved = interleaved;
    a.pos = positions;
    a.slots = slots;
    a.n_tok = n_tok;
    a.n_heads = S->d.n_heads;
    a.cache = static_cast<uint8_t *>(cache);
    a.page_stride = page_stride;
    a.n_pages = n_pages;
    a.page_shift = __builtin_ctz(static_cast<unsigned>(S->d.page_size));
    a.q_pe = static_cast<const uint8_t *>(q_pe);
    a.q_tok = q_tok_stride;
    a.q_head = q_head_stride;
    a.q_out = static_cast<uint8_t *>(q_out);
    a.err = S->err;
    OnDevice on(S->device);
    return launched(S, launch_append(a, S->d.half == COLI_HALF_BF16, static_cast<hipStream_t>(stream)), "append launch");
}

coli_status coli_latent_keep(coli_serve *S, void *cache, int64_t page_stride, int32_t n_pages, int32_t n_layers, int64_t layer_stride,
                             const int32_t *block_table, int64_t table_stride, int32_t table_cols, const int32_t *q_start,
                             const int32_t *kv_len, int32_t n_seq, int32_t n_tok, const int32_t *path, int64_t path_stride,
                             int32_t path_cols, void *stream) {
    NEED(S, "handle is NULL");
    CHECK(check_counts(S, n_tok, n_seq));
    CHECK(check_cache(S, cache, page_stride, n_pages));
    NEED(n_layers >= 0 && path_cols >= 0 && table_cols >= 0, "n_layers, path_cols and table_cols must be >= 0");
    NEED(layer_stride % 8 == 0, "layer_stride must be a multiple of 8 elements");
    if (n_seq == 0 || n_layers == 0 || path_cols == 0) return COLI_OK;
    NEED(block_table && q_start && kv_len && path, "NULL device pointer");
    KeepArgs a{};
    a.cache = view(S, cache, page_stride, n_pages, block_table, table_stride, table_cols);
    a.n_layers = n_layers;
    a.layer_stride = layer_stride;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.path = path;
    a.path_stride = path_stride;
    a.path_cols = path_cols;
    a.n_seq = n_seq;
    a.n_tok = n_tok;
    a.err = S->err;
    OnDevice on(S->device);
    return launched(S, launch_keep(a, static_cast<hipStream_t>(stream)), "keep launch");
}

coli_status coli_latent_plan(coli_serve *S, const int32_t *q_start, const int32_t *kv_len, int32_t n_seq, int32_t n_tok, void *stream) {
    NEED(S, "handle is NULL");
    CHECK(check_counts(S, n_tok, n_seq));
    if (n_seq > 0) NEED(q_start && kv_len, "NULL device pointer");
    OnDevice on(S->device);
    CHECK(launched(S, launch_decode_plan(S->plan, q_start, kv_len, n_seq, n_tok, S->d.n_heads, S->n_cu, S->err, static_cast<hipStream_t>(stream)),
                   "plan launch"));
    S->plan_tok = n_tok;
    S->plan_seq = n_seq;
    return COLI_OK;
}

coli_status coli_latent_decode(coli_serve *S, const void *q_lat, int64_t ql_tok_stride, int64_t ql_head_stride, const void *q_pe,
                               int64_t qp_tok_stride, int64_t qp_head_stride, const void *cache, int64_t page_stride, int32_t n_pages,
                               const int32_t *block_table, int64_t table_stride, int32_t table_cols, const uint64_t *tree_mask,
                               int32_t mask_words, float scale, int32_t n_tok, void *out, float *lse, void *stream) {
    NEED(S, "handle is NULL");
    if (S->plan_tok < 0) return fail(S, COLI_E_STATE, "no plan: coli_latent_plan comes first");
    NEED(n_tok == S->plan_tok, "n_tok %d differs from the plan's %d", n_tok, S->plan_tok);
    CHECK(check_cache(S, cache, page_stride, n_pages));
    NEED(std::isfinite(scale) && scale > 0.0f, "scale must be finite and > 0");
    NEED(table_cols >= 0, "table_cols must be >= 0");
    NEED(!tree_mask || mask_words >= 1, "mask_words %d must be >= 1", mask_words);
    if (n_tok == 0 || S->plan_seq == 0) return COLI_OK;
    NEED(q_lat && q_pe && block_table && out, "NULL device pointer");
    NEED(aligned(q_lat, 16) && aligned(q_pe, 16) && aligned(out, 16) && aligned(tree_mask, 8), "q_lat, q_pe and out must be 16-byte aligned, tree_mask 8-byte");
    NEED(ql_tok_stride % 8 == 0 && ql_head_stride % 8 == 0 && qp_tok_stride % 8 == 0 && qp_head_stride % 8 == 0, "strides must be multiples of 8 elements");
    DecodeArgs a{};
    a.q_lat = static_cast<const uint8_t *>(q_lat);
    a.q_pe = static_cast<const uint8_t *>(q_pe);
    a.ql_tok = ql_tok_stride;
    a.ql_head = ql_head_stride;
    a.qp_tok = qp_tok_stride;
    a.qp_head = qp_head_stride;
    a.cache = view(S, cache, page_stride, n_pages, block_table, table_stride, table_cols);
    a.mask = tree_mask;
    a.mask_words = mask_words;
    a.n_tok = n_tok;
    a.n_seq = S->plan_seq;
    a.n_heads = S->d.n_heads;
    a.scale = scale;
    a.out = static_cast<uint8_t *>(out);
    a.lse = lse;
    a.plan = S->plan;
    // A joined unit has two pieces at least.
    a.join_most = static_cast<int>(std::min<int64_t>(S->plan.join_cap, static_cast<int64_t>(n_tok) * S->d.n_heads / kTileRows + S->plan_seq));
    a.part = S->part;
    a.part_ml = S->part_ml;
    a.err = S->err;
    OnDevice on(S->device);
    return launched(S, launch_latent_decode(a, S->d.half == COLI_HALF_BF16, S->n_cu, static_cast<hipStream_t>(stream)), "decode launch");
}

coli_status coli_latent_prompt(coli_serve *S, const void *q, int64_t q_tok_stride, int64_t q_head_stride, const void *kv, int64_t kv_tok_stride,
                               int64_t kv_head_stride, const void *k_pe, int64_t pe_tok_stride, const int32_t *q_start, const int32_t *k_start,
                               int32_t n_seq, int32_t n_q, int32_t n_k, int32_t causal, float scale, void *out, float *lse, void *stream) {
    NEED(S, "handle is NULL");
    CHECK(check_counts(S, n_q, n_seq));
    NEED(n_k >= 0, "n_k %d must be >= 0", n_k);
    NEED(causal == 0 || causal == 1, "causal must be 0 or 1");
    NEED(std::isfinite(scale) && scale > 0.0f, "scale must be finite and > 0");
    if (n_q == 0 || n_seq == 0) return COLI_OK;
    NEED(q && q_start && k_start && out && (n_k == 0 || (kv && k_pe)), "NULL device pointer");
    NEED(aligned(q, 16) && aligned(kv, 16) && aligned(k_pe, 16) && aligned(out, 16), "q, kv, k_pe and out must be 16-byte aligned");
    NEED(q_tok_stride % 8 == 0 && q_head_stride % 8 == 0 && kv_tok_stride % 8 == 0 && kv_head_stride % 8 == 0 && pe_tok_stride % 8 == 0, "strides must be multiples of 8 elements");
    PromptArgs a{};
    a.q = static_cast<const uint8_t *>(q);
    a.kv = static_cast<const uint8_t *>(kv);
    a.k_pe = static_cast<const uint8_t *>(k_pe);
    a.q_tok = q_tok_stride;
    a.q_head = q_head_stride;
    a.kv_tok = kv_tok_stride;
    a.kv_head = kv_head_stride;
    a.pe_tok = pe_tok_stride;
    a.q_start = q_start;
    a.k_start = k_start;
    a.n_seq = n_seq;
    a.n_q = n_q;
    a.n_k = n_k;
    a.n_heads = S->d.n_heads;
    a.causal = causal;
    a.scale = scale;
    a.out = static_cast<uint8_t *>(out);
    a.lse = lse;
    a.part = S->part;
    a.part_ml = S->part_ml;
    // Parts of 128 rows that the slots hold: by their outputs, and by their statistics.
    a.part_cap = std::min(S->plan.slot_cap * (kTileRows * kLatent / 128) / S->d.v_dim, S->plan.slot_cap * (kTileRows * kSlotStats / 256));
    a.err = S->err;
    OnDevice on(S->device);
    return launched(S, launch_latent_prompt(a, S->d.half == COLI_HALF_BF16, S->d.nope, S->n_cu, static_cast<hipStream_t>(stream)), "prompt launch");
}

coli_status coli_draft_verify(coli_serve *S, const void *probs, int64_t probs_stride, const void *draft, int64_t draft_stride, int32_t kind,
                              int32_t vocab, const int32_t *tokens, const int32_t *parents, const int32_t *q_start, int32_t n_seq,
                              int32_t n_tok, const float *u, const float *race, int64_t race_stride, int32_t *path, int32_t path_cols,
                              int32_t *count, int32_t *next_tokens, void *stream) {
    NEED(S, "handle is NULL");
    CHECK(check_counts(S, n_tok, n_seq));
    NEED(kind == COLI_PROB_F32 || kind == COLI_PROB_BF16 || kind == COLI_PROB_F16, "kind must be COLI_PROB_F32, COLI_PROB_BF16 or COLI_PROB_F16");
    NEED(vocab >= 1 && vocab <= (1 << 27), "vocab %d must be in 1..2^27", vocab);
    NEED(path_cols >= 1, "path_cols %d must be >= 1", path_cols);
    if (n_seq == 0) return COLI_OK;
    if (n_seq > 65535) return fail(S, COLI_E_UNSUPPORTED, "n_seq %d: up to 65535 in one call", n_seq);
    NEED(q_start && path && count && next_tokens, "NULL device pointer");
    NEED(n_tok == 0 || (probs && tokens && u && race), "NULL device pointer");
    NEED(n_tok == 0 || (probs_stride >= vocab && race_stride >= vocab && (!draft || draft_stride >= vocab)), "row strides must be >= vocab");
    const size_t size = kind == COLI_PROB_F32 ? 4 : 2;
    NEED(aligned(probs, size) && aligned(draft, size), "probs and draft must be aligned to their elements");
    VerifyArgs a{};
    a.p = static_cast<const uint8_t *>(probs);
    a.q = static_cast<const uint8_t *>(draft);
    a.p_stride = probs_stride;
    a.q_stride = draft_stride;
    a.kind = kind;
    a.tokens = tokens;
    a.parents = parents;
    a.q_start = q_start;
    a.u = u;
    a.race = race;
    a.race_stride = race_stride;
    a.n_tok = n_tok;
    a.n_seq = n_seq;
    a.vocab = vocab;
    a.path_cols = path_cols;
    a.path = path;
    a.count = count;
    a.out_tokens = next_tokens;
    a.walk = S->walk;
    a.best = S->best;
    a.arrived = S->arrived;
    a.err = S->err;
    OnDevice on(S->device);
    return launched(S, launch_verify(a, S->n_cu, static_cast<hipStream_t>(stream)), "verify launch");
}

}  // extern "C"
