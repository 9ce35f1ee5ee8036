// The 8-bit paged KV cache: launch arguments of its kernels (page plans,
// rotary positions, append, attention).
//
// A pool holds n_pages pages.  A page is 64 consecutive tokens of one
// sequence: per kv head 64 rows of head_dim e4m3 codes for K and as many for
// V, [n_pages][n_kv][64][head_dim], and one fp32 scale each,
// [n_pages][n_kv]; a value is code * scale.  A sequence's block table row
// lists its pages in order.
#pragma once

#include "common.cuh"

namespace dfl {

constexpr int KV8_PAGE = 64;
constexpr size_t KV8_QUEUE_BYTES = 256;   // of an attention workspace, then its tickets, then partials
constexpr int KV8_TICKETS = 16384;        // tiles x kv heads of a call whose pages are split

struct PagesPlanArgs {
    const int* kv_len;
    const int* q_len;
    const int* free_pages;
    const int* n_free;
    int* table;
    int* row_start;
    int* positions;
    int* slots;
    int* kv_after;
    int* n_free_out;
    int S, free_cap, max_pages, rows;
};
int launch_pages_plan(const PagesPlanArgs& a, cudaStream_t s);

struct PagesTrimArgs {
    int* kv_len;
    const int* new_len;
    int* free_pages;
    int* n_free;
    int* table;
    int S, free_cap, max_pages;
};
int launch_pages_trim(const PagesTrimArgs& a, cudaStream_t s);

struct RopeTurnsArgs {
    int half, scaling;          // half = rotary_dim / 2
    double theta, factor, original_len, alpha, beta;
    unsigned long long* turns;
};
int launch_rope_turns(const RopeTurnsArgs& a, cudaStream_t s);

struct RopeHeads {
    const void* x;
    void* out;
    int heads;
    long long x_row, x_head, out_row, out_head;   // elements
};
struct RopeArgs {
    RopeHeads t[2];             // t[1].heads may be 0
    const unsigned long long* turns;
    const int* positions;
    int rows, head_dim, rotary, interleaved, dtype;
    float scale;
    int wide;                   // every row of every head is 16-byte aligned in whole units
};
int launch_rope(const RopeArgs& a, cudaStream_t s);

struct Kv8AppendArgs {
    const void* x[2];           // k, v
    long long row[2], head[2];  // element strides
    uint8_t* codes[2];
    float* scale[2];
    const int* slots;
    int rows, n_kv, head_dim, n_pages, dtype;
    int wide;                   // rows of x are 16-byte aligned
    int* err;
};
int launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t s);

struct Kv8AttnArgs {
    const void* q;
    void* out;
    float* lse;                 // [rows][n_q] or NULL
    long long q_row, q_head, out_row, out_head;
    const uint8_t* v_codes;
    const float* k_scale;
    const float* v_scale;
    const int* table;
    const int* kv_len;
    const int* row_start;
    int rows, S, n_q, n_kv, group, max_pages, n_pages, dtype;
    int causal, window;
    float scale_log2;           // softmax scale * log2(e)
    int split_cap;              // most splits of a tile's keys
    uint8_t caps[32];           // splits at most of a sequence with 2^b .. 2^(b+1) - 1 pages to read
    int tile, tile_log2;        // packed (row, q head) rows of an item
    float* part;                // [part_cap] partial tiles
    long long part_cap;
    int* queue;                 // [next item, CTAs done], zero between calls
    int* tickets;               // [tile slots][n_kv], zero between calls
    long long ticket_cap;
    int* err;
};

// Host: the kernel, split limit, workspace floats and tickets of an attention call.
enum : int { KV8_MMA = 0, KV8_TC_KEYS = 1, KV8_TC_ROWS = 2 };
struct Kv8AttnPlan {
    int form;                   // KV8_MMA, KV8_TC_KEYS or KV8_TC_ROWS
    int tile;
    int split_cap;
    uint8_t caps[32];
    long long part_cap, ticket_cap;
    size_t ticket_bytes, bytes;
};
Kv8AttnPlan kv8_attn_plan(int rows, int S, int n_q, int n_kv, int head_dim, int max_pages, int sms);
int launch_kv8_attention(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a,
                         int form, int head_dim, int sms, cudaStream_t s);
int launch_kv8_attention_tc(const CUtensorMap& k_map, const CUtensorMap& v_map, const Kv8AttnArgs& a,
                            int head_dim, int sms, cudaStream_t s);
struct Kv8WeighArgs {
    const void* q;
    const float* lse;           // [rows][n_q]
    long long q_row, q_head;
    const uint8_t* k_codes;
    const float* k_scale;
    const int* table;
    const int* kv_len;
    const int* row_start;
    const int* count;           // [S] or NULL
    float* weights;             // [n_pages][64]
    int rows, S, n_q, n_kv, group, max_pages, n_pages, dtype;
    int causal, window, observe, fresh;
    float scale_log2;
    int* err;
};
int launch_kv8_weigh(const Kv8WeighArgs& a, int head_dim, int sms, cudaStream_t s);
// The tcgen05 form: whether it is the faster one for a call's rows (and can take their strides), and its launch; q_map in
// boxes of 64 dims x group heads x (128 / group) rows.
bool kv8_weigh_by_tc(const Kv8WeighArgs& a);
int launch_kv8_weigh_tc(const CUtensorMap& q_map, const Kv8WeighArgs& a, int head_dim, int sms, cudaStream_t s);

constexpr int KV8_LAYERS = 32;  // of one launch: the kernel arguments hold their pools' addresses
struct Kv8MoveLayers {
    uint8_t* k_codes[KV8_LAYERS];
    uint8_t* v_codes[KV8_LAYERS];
    float* k_scale[KV8_LAYERS];
    float* v_scale[KV8_LAYERS];
    int n;
};
struct Kv8EvictArgs {
    const int* table;
    const int* kv_len;
    const float* weights;
    float* weights_out;         // may be weights
    const int* budget;
    int* new_len;
    int* dropped;               // [S] or NULL
    int* source;                // [S][max_pages * 64]
    int* from;                  // the same as slots
    int* first_moved;           // [S] first position that holds another than before; new_len: none
    int S, max_pages, n_pages, n_kv, keep_first, keep_last;
    int* err;
    int keys;                   // weights held in shared memory by the choice (set by the launch)
};
// `choose`: with the choice (the first launch of a call), else the move of more layers.
int launch_kv8_evict(const Kv8EvictArgs& a, const Kv8MoveLayers& l, bool choose, int head_dim, int sms, cudaStream_t s);

struct PagesShiftArgs {
    const int* positions;
    const int* row_start;
    int* dropped;
    int* out;
    int rows, S;
};
int launch_pages_shift(const PagesShiftArgs& a, cudaStream_t s);

// The largest dynamic shared memory, allowed once per kernel and device.
cudaError_t allow_smem(const void* kern);

}  // namespace dfl
