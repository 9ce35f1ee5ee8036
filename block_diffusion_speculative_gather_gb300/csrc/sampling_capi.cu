// C entry points of sampled decoding: argument checks and launches.

#include <cstring>

#include "capi_internal.cuh"
#include "gemm.cuh"
#include "sampling.cuh"

using namespace dfl;

namespace {

constexpr int MAX_ROWS = 1 << 30;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int launched(int e, const char* what) {
    return e ? report_error(DFLASH_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString((cudaError_t)e)) : DFLASH_OK;
}

int pending() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DFLASH_OK
                            : report_error(DFLASH_ERR_CUDA, "a CUDA error was pending before this call: %s",
                                           cudaGetErrorString(e));
}

int units_of(int vocab) { return (vocab + VERIFY_UNIT - 1) / VERIFY_UNIT; }

int sm_count(int* sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return e == cudaSuccess ? DFLASH_OK : report_error(DFLASH_ERR_CUDA, "SM count: %s", cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int dflash_probs(const void* logits, int64_t logits_row, int32_t dtype, const float* temperature, const float* min_p,
                 int32_t rows, int32_t vocab, float* probs, int64_t probs_row, dflash_stream_t stream) {
    if (dtype != DFLASH_F32 && dtype != DFLASH_BF16 && dtype != DFLASH_F16)
        return report_error(DFLASH_ERR_ARG, "dtype %d: F32, BF16 or F16", dtype);
    if (rows < 0 || rows > MAX_ROWS || vocab < 1 || vocab > MAX_ROWS)
        return report_error(DFLASH_ERR_ARG, "rows %d vocab %d out of range", rows, vocab);
    if (rows == 0) return DFLASH_OK;
    if (!logits || !temperature || !probs) return report_error(DFLASH_ERR_ARG, "NULL argument");
    if (!aligned(logits, dtype == DFLASH_F32 ? 4 : 2) || !aligned(probs, 4) || !aligned(temperature, 4) ||
        !aligned(min_p, 4))
        return report_error(DFLASH_ERR_ARG, "misaligned rows");
    if (rows > 1 && (probs_row < vocab || logits_row < 0))
        return report_error(DFLASH_ERR_ARG, "probs_row %lld (vocab %d): rows of probs overlap; logits_row %lld",
                            (long long)probs_row, vocab, (long long)logits_row);
    if (logits == probs && (dtype != DFLASH_F32 || (rows > 1 && logits_row != probs_row)))
        return report_error(DFLASH_ERR_ARG, "in place: fp32 logits with probs' rows");
    if (const int r = pending()) return r;
    ProbsArgs a{logits, logits_row, probs_row, temperature, min_p, probs, rows, vocab,
                dtype == DFLASH_F32 ? 0 : (dtype == DFLASH_BF16 ? 1 : 2)};
    int sms = 0;
    if (const int r = sm_count(&sms)) return r;
    return launched(launch_probs(a, sms, reinterpret_cast<cudaStream_t>(stream)), "probabilities");
}

int dflash_selftest_exchange(const float* logits, const float* temperature, int32_t rows, int32_t vocab, float* probs,
                             int32_t stays, int32_t word, int32_t row, int64_t limit_ns, dflash_stream_t stream) {
    if (!logits || !temperature || !probs || !aligned(logits, 16) || !aligned(probs, 16) || !aligned(temperature, 4))
        return report_error(DFLASH_ERR_ARG, "NULL or misaligned argument");
    if (rows < 1 || rows > 4096 || vocab < 4 || vocab > SELFTEST_VOCAB || vocab % 4 || word < 0 || word > 1 || row < 0 ||
        limit_ns < 1 || limit_ns > 1000000000)
        return report_error(DFLASH_ERR_ARG, "rows %d (1 to 4096) vocab %d (4 to %d, by 4) word %d row %d limit_ns %lld (to 1 s)",
                            rows, vocab, SELFTEST_VOCAB, word, row, (long long)limit_ns);
    if (const int r = pending()) return r;
    ProbsArgs a{logits, vocab, vocab, temperature, nullptr, probs, rows, vocab, 0, row, word, (unsigned long long)limit_ns};
    return launched(launch_probs_selftest(a, stays != 0, reinterpret_cast<cudaStream_t>(stream)), "probabilities' self-test");
}

size_t dflash_verify_workspace_bytes(int32_t S, int32_t vocab) {
    if (S < 1 || S > VERIFY_MAX_SEQS || vocab < 1 || vocab > VERIFY_MAX_VOCAB) {
        report_error(DFLASH_ERR_CONFIG, "S %d (1 to %d) vocab %d (1 to 2^24)", S, VERIFY_MAX_SEQS, vocab);
        return 0;
    }
    return VERIFY_TICKET_BYTES + (size_t)S * units_of(vocab) * sizeof(float2);
}

int dflash_verify_drafts(const dflash_drafts* d, void* workspace, size_t workspace_bytes, int32_t* err,
                         dflash_stream_t stream) {
    if (!d || !workspace || !aligned(workspace, 256) || !err || !aligned(err, 8))
        return report_error(DFLASH_ERR_ARG, "NULL or misaligned argument");
    const size_t need = dflash_verify_workspace_bytes(d->S, d->vocab);
    if (need == 0) return DFLASH_ERR_CONFIG;
    if (d->rows < 0 || d->rows > MAX_ROWS || d->probs_row < 0 || d->draft_row < 0)
        return report_error(DFLASH_ERR_ARG, "rows %d probs_row %lld draft_row %lld out of range", d->rows,
                            (long long)d->probs_row, (long long)d->draft_row);
    if (!d->row_start || !d->n_tokens || !d->new_len != !d->kv_len)
        return report_error(DFLASH_ERR_ARG, "NULL row_start or n_tokens, or one of kv_len and new_len");
    if (d->rows > 0 && (!d->probs || !d->ids || !d->uniform || !d->tokens))
        return report_error(DFLASH_ERR_ARG, "NULL argument");
    if (d->rows > 0 && d->tokens == d->ids) return report_error(DFLASH_ERR_ARG, "tokens is ids: both are needed");
    if (!aligned(d->probs, 4) || !aligned(d->draft_probs, 4)) return report_error(DFLASH_ERR_ARG, "misaligned rows");
    if (workspace_bytes < need) return report_error(DFLASH_ERR_ARG, "workspace %zu < %zu", workspace_bytes, need);
    if (const int r = pending()) return r;
    VerifyArgs a;
    memset(&a, 0, sizeof a);
    a.p = d->probs;
    a.q = d->draft_probs;
    a.p_row = d->probs_row;
    a.q_row = d->draft_row;
    a.ids = d->ids;
    a.u = d->uniform;
    a.row_start = d->row_start;
    a.kv_len = d->kv_len;
    a.tokens = d->tokens;
    a.n_tokens = d->n_tokens;
    a.new_len = d->new_len;
    a.tickets = static_cast<int*>(workspace);
    a.part = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + VERIFY_TICKET_BYTES);
    a.rows = d->rows;
    a.vocab = d->vocab;
    a.S = d->S;
    a.units = units_of(d->vocab);
    a.wide = d->vocab % 4 == 0 && aligned(d->probs, 16) && aligned(d->draft_probs, 16) && d->probs_row % 4 == 0 &&
             d->draft_row % 4 == 0;
    a.err = err;
    int sms = 0;
    if (const int r = sm_count(&sms)) return r;
    return launched(launch_verify_drafts(a, sms, reinterpret_cast<cudaStream_t>(stream)), "draft verification");
}

}  // extern "C"
