// Sampled decoding: launch arguments of the probability and verification kernels.
#pragma once

#include "common.cuh"

namespace dfl {

struct ProbsArgs {
    const void* x;              // logits [rows][vocab]
    long long x_row, p_row;     // elements between rows
    const float* temperature;   // [rows]
    const float* min_p;         // [rows] or NULL
    float* p;
    int rows, vocab, dtype;     // dtype 0 fp32, 1 bf16, 2 f16
    // of the self-test's kernels alone: the row and exchange without one CTA's word, how long waits last
    int quiet_row, quiet;
    unsigned long long limit_ns;
};
int launch_probs(const ProbsArgs& a, int sms, cudaStream_t s);
constexpr int SELFTEST_VOCAB = 4096;     // tokens that clusters of two hold, four a thread
// fp32 rows of whole aligned vectors, by clusters of two: one a row, or (`stays`) one for all.
int launch_probs_selftest(const ProbsArgs& a, bool stays, cudaStream_t s);

constexpr int VERIFY_MAX_SEQS = 65535;
constexpr int VERIFY_MAX_VOCAB = 1 << 24;
constexpr int VERIFY_UNIT = 1024;        // tokens that a warp sums at a time
// tickets first, at the same place in every call, so that calls of different
// shapes can share a workspace: none's sums lie where another counts
constexpr size_t VERIFY_TICKET_BYTES = 65536 * sizeof(int);

struct VerifyArgs {
    const float* p;             // [rows][vocab]
    const float* q;             // [rows][vocab] or NULL: drafts are certain
    long long p_row, q_row;
    const int* ids;
    const float* u;
    const int* row_start;
    const int* kv_len;          // [S] or NULL
    int* tokens;
    int* n_tokens;
    int* new_len;               // [S] or NULL
    int* tickets;               // [S], zero between calls
    float2* part;               // [S][units] sums of weights, each as two fp32 numbers
    int rows, vocab, S, units;
    int wide;                   // rows of p and q are 16-byte aligned
    int* err;
};
int launch_verify_drafts(const VerifyArgs& a, int sms, cudaStream_t s);

}  // namespace dfl
