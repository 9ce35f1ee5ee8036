// C entry points of the 8-bit paged KV cache and of rotary positions:
// argument checks, tensor maps and launches.

#include <cmath>
#include <cstring>

#include "capi_internal.cuh"
#include "gemm.cuh"
#include "kv8.cuh"

using namespace dfl;

namespace {

constexpr int KV8_MAX_SEQS = 4096;        // a lane of an attention CTA's finding warp scans S / 32 of them
constexpr int KV8_MAX_PAGES = 1 << 25;    // slots are int32
constexpr int MAX_COUNT = 1 << 30;        // rows or sequences: sums of two of them, and a step beyond, are int32

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t size_of(int dtype) { return dtype == DFLASH_F32 ? 4 : 2; }

int launched(int e, const char* what) {
    return e ? report_error(DFLASH_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString((cudaError_t)e)) : DFLASH_OK;
}

int pending() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DFLASH_OK
                            : report_error(DFLASH_ERR_CUDA, "a CUDA error was pending before this call: %s",
                                           cudaGetErrorString(e));
}

int check_cache(const dflash_kv8_cache* c) {
    if (!c || !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale)
        return report_error(DFLASH_ERR_ARG, "NULL cache buffer");
    if (c->head_dim != 64 && c->head_dim != 128)
        return report_error(DFLASH_ERR_CONFIG, "head_dim %d: 64 or 128", c->head_dim);
    if (c->n_kv < 1 || c->n_kv > 1024 || c->n_pages < 1 ||
        (long long)c->n_pages * c->n_kv >= KV8_MAX_PAGES)
        return report_error(DFLASH_ERR_CONFIG, "n_pages %d n_kv %d: at least 1, n_kv at most 1024, product below 2^25",
                            c->n_pages, c->n_kv);
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return report_error(DFLASH_ERR_ARG, "misaligned cache buffer");
    return DFLASH_OK;
}

int sm_count(int* sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return e == cudaSuccess ? DFLASH_OK : report_error(DFLASH_ERR_CUDA, "SM count: %s", cudaGetErrorString(e));
}

// Bounds of an attention call's shape, shared with its workspace size.
int check_attn_shape(int rows, int S, int n_q, int n_kv, int head_dim, int max_pages) {
    if (head_dim != 64 && head_dim != 128)
        return report_error(DFLASH_ERR_CONFIG, "head_dim %d: 64 or 128", head_dim);
    if (n_kv < 1 || n_q < n_kv || n_q % n_kv || n_q / n_kv > 16 || n_q > 1024)
        return report_error(DFLASH_ERR_CONFIG, "n_q %d n_kv %d: n_q a multiple of n_kv, at most 16 per kv head", n_q, n_kv);
    if (S < 1 || S > KV8_MAX_SEQS)
        return report_error(DFLASH_ERR_CONFIG, "%d sequences: 1 to %d", S, KV8_MAX_SEQS);
    if (rows < 0 || max_pages < 1 || max_pages >= KV8_MAX_PAGES)
        return report_error(DFLASH_ERR_ARG, "rows %d max_pages %d out of range", rows, max_pages);
    // items are counted in int32
    if (((long long)rows * n_q + 16LL * S * n_kv) * 4 >= (1LL << 31))
        return report_error(DFLASH_ERR_CONFIG, "rows %d x n_q %d: too many for one call", rows, n_q);
    return DFLASH_OK;
}

}  // namespace

extern "C" {

int dflash_pages_plan(const int32_t* kv_len, const int32_t* q_len, int32_t S, const int32_t* free_pages,
                      int32_t free_cap, const int32_t* n_free, int32_t* table, int32_t max_pages, int32_t rows,
                      int32_t* row_start, int32_t* positions, int32_t* slots, int32_t* kv_after,
                      int32_t* n_free_out, dflash_stream_t stream) {
    if (!kv_len || !q_len || !n_free || !table || !row_start || !kv_after || !n_free_out)
        return report_error(DFLASH_ERR_ARG, "NULL argument");
    if (S < 1 || S > MAX_COUNT || free_cap < 0 || max_pages < 1 || max_pages >= KV8_MAX_PAGES || rows < 0 ||
        rows > MAX_COUNT)
        return report_error(DFLASH_ERR_ARG, "S %d free_cap %d max_pages %d rows %d out of range", S, free_cap,
                            max_pages, rows);
    if ((free_cap && !free_pages) || (rows && (!positions || !slots)))
        return report_error(DFLASH_ERR_ARG, "NULL argument");
    if (const int r = pending()) return r;
    PagesPlanArgs a{kv_len, q_len, free_pages, n_free, table, row_start, positions, slots,
                    kv_after, n_free_out, S, free_cap, max_pages, rows};
    return launched(launch_pages_plan(a, reinterpret_cast<cudaStream_t>(stream)), "page plan");
}

int dflash_pages_trim(int32_t* kv_len, const int32_t* new_len, int32_t S, int32_t* free_pages, int32_t free_cap,
                      int32_t* n_free, int32_t* table, int32_t max_pages, dflash_stream_t stream) {
    if (!kv_len || !new_len || !n_free || !table || (free_cap && !free_pages))
        return report_error(DFLASH_ERR_ARG, "NULL argument");
    if (S < 1 || S > MAX_COUNT || free_cap < 0 || max_pages < 1 || max_pages >= KV8_MAX_PAGES)
        return report_error(DFLASH_ERR_ARG, "S %d free_cap %d max_pages %d out of range", S, free_cap, max_pages);
    if (const int r = pending()) return r;
    PagesTrimArgs a{kv_len, new_len, free_pages, n_free, table, S, free_cap, max_pages};
    return launched(launch_pages_trim(a, reinterpret_cast<cudaStream_t>(stream)), "page trim");
}

static int check_rope(const dflash_rope_config* c) {
    if (!c) return report_error(DFLASH_ERR_ARG, "NULL rope config");
    if (c->rotary_dim < 2 || c->rotary_dim % 2 || c->rotary_dim > 1024)
        return report_error(DFLASH_ERR_CONFIG, "rotary_dim %d: even, 2 to 1024", c->rotary_dim);
    if (!(c->theta > 1.0) || !std::isfinite(c->theta) || !std::isfinite(c->scale))
        return report_error(DFLASH_ERR_CONFIG, "theta %g (above 1) or scale %g", c->theta, (double)c->scale);
    if (c->scaling < DFLASH_ROPE_NONE || c->scaling > DFLASH_ROPE_PARTS)
        return report_error(DFLASH_ERR_CONFIG, "scaling %d", c->scaling);
    if (c->scaling != DFLASH_ROPE_NONE && (!(c->factor >= 1.0) || !std::isfinite(c->factor)))
        return report_error(DFLASH_ERR_CONFIG, "factor %g: at least 1", c->factor);
    if (c->scaling == DFLASH_ROPE_PARTS && (c->original_len < 1 || !(c->beta > c->alpha) || !std::isfinite(c->beta) ||
                                            !std::isfinite(c->alpha)))
        return report_error(DFLASH_ERR_CONFIG, "original_len %d alpha %g beta %g", c->original_len, c->alpha, c->beta);
    return DFLASH_OK;
}

int dflash_rope_turns(const dflash_rope_config* cfg, uint64_t* turns, dflash_stream_t stream) {
    if (const int r = check_rope(cfg)) return r;
    if (!turns || !aligned(turns, 8)) return report_error(DFLASH_ERR_ARG, "turns NULL or misaligned");
    if (const int r = pending()) return r;
    RopeTurnsArgs a{cfg->rotary_dim / 2, cfg->scaling, cfg->theta, cfg->factor, (double)cfg->original_len,
                    cfg->alpha, cfg->beta, reinterpret_cast<unsigned long long*>(turns)};
    return launched(launch_rope_turns(a, reinterpret_cast<cudaStream_t>(stream)), "rope turns");
}

int dflash_rope(const dflash_rope_config* cfg, const uint64_t* turns, const int32_t* positions, int32_t rows,
                int32_t head_dim, int32_t dtype, const dflash_heads* a, const dflash_heads* b,
                dflash_stream_t stream) {
    if (const int r = check_rope(cfg)) return r;
    if (!turns || !a || (rows > 0 && !positions)) return report_error(DFLASH_ERR_ARG, "NULL argument");
    if (dtype != DFLASH_F32 && dtype != DFLASH_BF16 && dtype != DFLASH_F16)
        return report_error(DFLASH_ERR_ARG, "dtype %d: F32, BF16 or F16", dtype);
    if (rows < 0 || rows > MAX_COUNT || head_dim < cfg->rotary_dim || head_dim > 1024)
        return report_error(DFLASH_ERR_ARG, "rows %d head_dim %d (rotary_dim %d to 1024)", rows, head_dim,
                            cfg->rotary_dim);
    const size_t es = size_of(dtype);
    const int V = (int)(16 / es);
    RopeArgs r;
    memset(&r, 0, sizeof r);
    r.wide = (cfg->interleaved ? cfg->rotary_dim : cfg->rotary_dim / 2) % V == 0 &&
             (head_dim - cfg->rotary_dim) % V == 0;
    const dflash_heads* in[2] = {a, b};
    for (int i = 0; i < 2; ++i) {
        const dflash_heads* t = in[i];
        if (!t) continue;
        if (t->heads < 0 || t->heads > 65536) return report_error(DFLASH_ERR_ARG, "heads %d", t->heads);
        if (t->heads == 0) continue;
        if (rows > 0 && (!t->x || !t->out)) return report_error(DFLASH_ERR_ARG, "NULL rows");
        if (!aligned(t->x, es) || !aligned(t->out, es)) return report_error(DFLASH_ERR_ARG, "misaligned rows");
        if (rows > 0 && t->x == t->out && (t->x_row != t->out_row || t->x_head != t->out_head))
            return report_error(DFLASH_ERR_ARG, "in place with two sets of strides");
        r.t[i] = RopeHeads{t->x, t->out, t->heads, t->x_row, t->x_head, t->out_row, t->out_head};
        r.wide = r.wide && aligned(t->x, 16) && aligned(t->out, 16) && t->x_row % V == 0 && t->x_head % V == 0 &&
                 t->out_row % V == 0 && t->out_head % V == 0;
    }
    if (rows == 0 || r.t[0].heads + r.t[1].heads == 0) return DFLASH_OK;
    if (const int e = pending()) return e;
    r.turns = reinterpret_cast<const unsigned long long*>(turns);
    r.positions = positions;
    r.rows = rows;
    r.head_dim = head_dim;
    r.rotary = cfg->rotary_dim;
    r.interleaved = cfg->interleaved != 0;
    r.dtype = dtype == DFLASH_F32 ? 0 : (dtype == DFLASH_BF16 ? 1 : 2);
    r.scale = cfg->scale;
    return launched(launch_rope(r, reinterpret_cast<cudaStream_t>(stream)), "rope");
}

int dflash_kv8_append(const dflash_kv8_cache* cache, const void* k, int64_t k_row, int64_t k_head, const void* v,
                      int64_t v_row, int64_t v_head, int32_t dtype, int32_t rows, const int32_t* slots,
                      int32_t* err, dflash_stream_t stream) {
    if (const int r = check_cache(cache)) return r;
    if (dtype != DFLASH_F32 && dtype != DFLASH_BF16 && dtype != DFLASH_F16)
        return report_error(DFLASH_ERR_ARG, "dtype %d: F32, BF16 or F16", dtype);
    if (rows < 0 || rows > MAX_COUNT || !err || !aligned(err, 8))
        return report_error(DFLASH_ERR_ARG, "rows %d or err", rows);
    if (rows == 0) return DFLASH_OK;
    if (!k || !v || !slots) return report_error(DFLASH_ERR_ARG, "NULL argument");
    const size_t es = size_of(dtype);
    if (!aligned(k, es) || !aligned(v, es)) return report_error(DFLASH_ERR_ARG, "misaligned rows");
    if (const int r = pending()) return r;
    const int V = (int)(16 / es);
    Kv8AppendArgs a{{k, v}, {k_row, v_row}, {k_head, v_head}, {cache->k_codes, cache->v_codes},
                    {cache->k_scale, cache->v_scale}, slots, rows, cache->n_kv, cache->head_dim, cache->n_pages,
                    dtype == DFLASH_F32 ? 0 : (dtype == DFLASH_BF16 ? 1 : 2),
                    aligned(k, 16) && aligned(v, 16) && k_row % V == 0 && k_head % V == 0 && v_row % V == 0 &&
                        v_head % V == 0,
                    err};
    return launched(launch_kv8_append(a, reinterpret_cast<cudaStream_t>(stream)), "cache append");
}

size_t dflash_kv8_workspace_bytes(int32_t rows, int32_t S, int32_t n_q, int32_t n_kv, int32_t head_dim,
                                  int32_t max_pages) {
    if (check_attn_shape(rows, S, n_q, n_kv, head_dim, max_pages)) return 0;
    // the splits follow the current device's SM count (without a device: the
    // part this library is made for)
    int sms = 0;
    if (sm_count(&sms)) {
        cudaGetLastError();
        sms = 152;
    }
    return kv8_attn_plan(rows, S, n_q, n_kv, head_dim, max_pages, sms > 256 ? 256 : sms).bytes;
}

int dflash_kv8_attention(const dflash_kv8_cache* cache, const dflash_kv8_query* q, void* workspace,
                         size_t workspace_bytes, int32_t* err, dflash_stream_t stream) {
    if (const int r = check_cache(cache)) return r;
    if (!q || !workspace || !err || !aligned(err, 8)) return report_error(DFLASH_ERR_ARG, "NULL argument");
    if (const int r = check_attn_shape(q->rows, q->S, q->n_q, cache->n_kv, cache->head_dim, q->max_pages)) return r;
    if (q->dtype != DFLASH_BF16 && q->dtype != DFLASH_F16)
        return report_error(DFLASH_ERR_ARG, "dtype %d: BF16 or F16", q->dtype);
    if (!(q->scale > 0.f) || !std::isfinite(q->scale * 1.4426950408889634f) || q->window < 0)
        return report_error(DFLASH_ERR_ARG, "scale %g (above 0) window %d", (double)q->scale, q->window);
    if (q->rows == 0) return DFLASH_OK;
    if (!q->q || !q->out || !q->table || !q->kv_len || !q->row_start) return report_error(DFLASH_ERR_ARG, "NULL argument");
    if (!aligned(q->q, 16) || !aligned(q->out, 16) || q->q_row % 8 || q->q_head % 8 || q->out_row % 8 ||
        q->out_head % 8 || !aligned(workspace, 256))
        return report_error(DFLASH_ERR_ARG, "q, out: 16-byte aligned rows of every head; workspace: 256");
    int sms = 0;
    if (const int r = sm_count(&sms)) return r;
    if (sms > 256) sms = 256;
    const Kv8AttnPlan plan = kv8_attn_plan(q->rows, q->S, q->n_q, cache->n_kv, cache->head_dim, q->max_pages, sms);
    if (workspace_bytes < plan.bytes)
        return report_error(DFLASH_ERR_ARG, "workspace %zu < %zu", workspace_bytes, plan.bytes);
    if (const int r = pending()) return r;
    CUtensorMap k_map, v_map;
    const int hd = cache->head_dim;
    const uint64_t tile_rows = (uint64_t)cache->n_pages * cache->n_kv * KV8_PAGE;
    const CUtensorMapSwizzle swz = hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    int r = encode_map(&k_map, cache->k_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, hd, tile_rows, hd, KV8_PAGE, swz);
    if (!r) r = encode_map(&v_map, cache->v_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, hd, tile_rows, hd, KV8_PAGE, swz);
    if (r) return r;
    Kv8AttnArgs a;
    memset(&a, 0, sizeof a);
    a.q = q->q;
    a.out = q->out;
    a.lse = q->lse;
    a.q_row = q->q_row;
    a.q_head = q->q_head;
    a.out_row = q->out_row;
    a.out_head = q->out_head;
    a.v_codes = cache->v_codes;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.table = q->table;
    a.kv_len = q->kv_len;
    a.row_start = q->row_start;
    a.rows = q->rows;
    a.S = q->S;
    a.n_q = q->n_q;
    a.n_kv = cache->n_kv;
    a.group = q->n_q / cache->n_kv;
    a.max_pages = q->max_pages;
    a.n_pages = cache->n_pages;
    a.dtype = q->dtype == DFLASH_BF16 ? 1 : 2;
    a.causal = q->causal != 0;
    a.window = q->window;
    a.scale_log2 = q->scale * 1.4426950408889634f;
    a.split_cap = plan.split_cap;
    memcpy(a.caps, plan.caps, sizeof a.caps);
    a.tile = plan.tile;
    while ((1 << a.tile_log2) < plan.tile) ++a.tile_log2;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.queue = reinterpret_cast<int*>(ws);
    a.tickets = reinterpret_cast<int*>(ws + KV8_QUEUE_BYTES);
    a.ticket_cap = plan.ticket_cap;
    a.part = reinterpret_cast<float*>(ws + KV8_QUEUE_BYTES + plan.ticket_bytes);
    a.part_cap = plan.part_cap;
    a.err = err;
    return launched(launch_kv8_attention(k_map, v_map, a, plan.form, hd, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "cache attention");
}

}  // extern "C"
