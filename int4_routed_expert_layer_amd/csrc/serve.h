// serve.h -- shared declarations of the serving operators beside the expert
// layer: the latent cache, latent attention (absorbed and expanded) and the
// verification of drafted tokens (not part of the ABI).
#pragma once

#include "internal.h"

namespace coli {

constexpr int kLatent = 512;             // latent values of one cached token: keys and values of every head
constexpr int kRope = 64;                // its rotary key values
constexpr int kCacheRow = kLatent + kRope;
constexpr int kRowBytes = 2 * kCacheRow;
// A row of an 8-bit cache: the latent values in e4m3, the rotary ones in 16 bits, a
// scale's exponent (biased by 127) for each 32 latent values.
constexpr int kScaleGroup = 32;
constexpr int kRow8Rope = kLatent, kRow8Scales = kLatent + 2 * kRope;
constexpr int kRow8Bytes = kRow8Scales + kLatent / kScaleGroup;
constexpr int kPrefixEntries = 1024;     // sequences and groups of a plan whose groups share prefixes
constexpr int kBeamMost = 64;            // beams of a group, and continuations kept of one
constexpr int kTileKeys = 64;            // cached tokens per attention tile
constexpr int kTileRows = 64;            // (token, head) rows per absorbed-attention item
constexpr int kVerifyMaxNodes = 1024;    // drafted nodes of one sequence

// Device error flags of a serve handle (coli_serve_device_errors).
constexpr int32_t kErrSeq = 1;        // a sequence's bounds are outside the call's tokens
constexpr int32_t kErrPage = 2;       // a page number, slot or position outside the cache or tables
constexpr int32_t kErrDraft = 4;      // a drafted node, token or path outside its sequence or vocabulary
constexpr int32_t kErrNoMass = 8;     // no token of a row has a positive probability

// One piece of absorbed attention: 64 rows of one sequence against the key
// tiles [t0, t1).  slot >= 0: a partial result, joined with the other pieces
// of its rows afterwards.  Items are laid out in rounds of one per workgroup;
// n == 0 is a place without one.
struct alignas(32) DecodeItem {
    int32_t q0, n, len, seq;   // first token, tokens and cached length of the sequence; seq | kItemMore: rounds follow;
                               // | kItemPrefix: a group's tokens and prefix, seq its first sequence
    int32_t row0, t0, t1, slot;
};
constexpr int32_t kItemMore = 1 << 30, kItemPrefix = 1 << 29;
// Rows whose pieces are joined: `rows` output rows from out_row, the partials slot0 ..
// slot0 + split - 1.  split | kJoinGroup: they are a group's and the partials those of its
// prefix; each row has others, found by its token's record: of unit i of the sequence
// whose first row is row0, slot0 + i split ...
struct alignas(16) JoinUnit {
    int32_t out_row, rows, slot0, split;
};
constexpr int32_t kJoinGroup = 1 << 30;
typedef int32_t TokenRecord __attribute__((ext_vector_type(4)));   // slot0, split, row0
constexpr int kRecords = 65536;          // tokens of a plan with prefixes, whose rows (64 to a unit) have to find room
struct DecodePlan {
    int32_t *head;             // [4] join units, the most pieces of one, tokens, sequences
    DecodeItem *items;
    JoinUnit *joins;
    TokenRecord *records;      // [min(max_tokens, kRecords)]
    int32_t *seq;              // [max_seqs x 4] scratch of the planning
    int item_cap, join_cap, slot_cap;
};

struct CacheView {
    uint8_t *base;
    int64_t page_bytes;        // from one page to the next
    int n_pages, page_shift;
    const int32_t *table;      // [n_seq x table_cols] page numbers
    int64_t table_stride;
    int table_cols;
};

struct DecodeArgs {
    const uint8_t *q_lat, *q_pe;
    int64_t ql_tok, ql_head, qp_tok, qp_head;   // strides in elements
    CacheView cache;
    const uint64_t *mask;      // [n_tok x mask_words] ancestor bits, or NULL for a chain
    int mask_words;
    int n_tok, n_seq, n_heads;
    float scale;
    uint8_t *out;              // [n_tok x n_heads x 512]
    float *lse;                // [n_tok x n_heads] or NULL
    DecodePlan plan;
    int join_most;             // at least the plan's join units
    float *part;               // [slot_cap x 64 x 512], in the order of join_kernel's blocks
    float *part_ml;            // [slot_cap x 64 x 2], with room for part_cap of the prompts
    int32_t *err;
};

struct PromptArgs {
    const uint8_t *q, *kv, *k_pe;
    int64_t q_tok, q_head, kv_tok, kv_head, pe_tok;   // strides in elements
    const int32_t *q_start, *k_start;
    int n_seq, n_q, n_k, n_heads, causal;
    float scale;
    uint8_t *out;              // [n_q x n_heads x v]
    float *lse;                // [n_q x n_heads] or NULL
    float *part;               // [part_cap x 128 x v], in the order of join_parts_kernel's blocks
    float *part_ml;            // [part_cap x 128 x 2]
    int part_cap, split;       // split: set by the launcher, parts per tile at most
    int32_t *err;
};

struct AppendArgs {
    const uint8_t *c, *weight;
    int64_t c_stride;
    float eps;
    const float *cos_t, *sin_t;
    int n_pos, interleaved;
    const int32_t *pos;
    const int64_t *slots;
    int n_tok, n_heads;
    uint8_t *cache;
    int64_t page_bytes;
    int n_pages, page_shift;
    const uint8_t *q_pe;       // or NULL
    int64_t q_tok, q_head;
    uint8_t *q_out;
    int32_t *err;
};

struct KeepArgs {
    CacheView cache;
    int n_layers;
    int64_t layer_bytes;
    const int32_t *q_start, *kv_len, *path;
    int64_t path_stride;
    int path_cols, n_seq, n_tok;
    int32_t *err;
};

struct ReadArgs {
    CacheView cache;
    const int32_t *first, *k_start;   // first may be NULL
    int n_seq, n_rows;
    uint8_t *out;              // [n_rows x 576]
    int64_t out_stride;        // elements
    int32_t *err;
};

struct ReorderArgs {
    CacheView cache;
    int n_layers;
    int64_t layer_bytes;
    const int32_t *kv_len, *parents;   // [n_groups x beams]
    int n_groups, beams;
    int32_t *out_table;
    int64_t out_stride;
    int32_t *err;
};

struct SelectArgs {
    const uint8_t *logits;     // [n_groups x beams x vocab] rows
    int64_t stride;            // elements
    int kind;                  // coli_prob
    int vocab, n_groups, beams, keep;
    const float *scores;       // [n_groups x beams]
    float *out_scores;         // [n_groups x keep]
    int32_t *parents, *tokens;
    uint64_t *best;            // scratch: [rows of a launch x chunks x keep]
    float2 *sums;              // [rows of a launch x chunks] maximum and sum
    int64_t best_cap, sums_cap;
    int32_t *err;
};

struct VerifyArgs {
    const uint8_t *p, *q;      // [n_tok x vocab], q may be NULL
    int64_t p_stride, q_stride;
    int kind;                  // coli_prob
    const int32_t *tokens, *parents;   // parents NULL: chains
    const int32_t *q_start;
    const float *u, *race;
    int64_t race_stride;
    int n_tok, n_seq, vocab, path_cols;
    int32_t *path, *count, *out_tokens;
    int32_t *walk;             // [n_seq x 4] final node, its refused children, residual factor (float)
    uint64_t *best;            // [n_seq x 2] zero at rest
    int32_t *arrived;          // [n_seq] zero at rest
    int32_t *err;
};

hipError_t launch_append(const AppendArgs &a, bool bf16, bool cache8, hipStream_t s);
hipError_t launch_keep(const KeepArgs &a, bool cache8, hipStream_t s);
hipError_t launch_read(const ReadArgs &a, bool bf16, bool cache8, hipStream_t s);
hipError_t launch_reorder(const ReorderArgs &a, bool cache8, hipStream_t s);
hipError_t launch_select(const SelectArgs &a, int n_cu, hipStream_t s);
hipError_t launch_decode_plan(const DecodePlan &p, const int32_t *q_start, const int32_t *kv_len, int n_seq, int n_tok,
                              int n_heads, int n_cu, const int32_t *group_start, const int32_t *prefix_len, int n_groups, int32_t *err,
                              hipStream_t s);
hipError_t launch_latent_decode(const DecodeArgs &a, bool bf16, bool cache8, bool prefixes, int n_cu, hipStream_t s);
hipError_t launch_latent_prompt(PromptArgs a, bool bf16, int nope, int n_cu, hipStream_t s);
hipError_t launch_verify(const VerifyArgs &a, int n_cu, hipStream_t s);

// abi.hip: device memory under the library's allocation book and cap.
hipError_t book_alloc(void **p, size_t n);
bool book_fits(size_t n);
void book_free(void *p);

}  // namespace coli
