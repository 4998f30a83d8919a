// dsa_paged.cuh -- what the append and the attention over the paged cache
// share: the batch as the kernels see it, and the handle.  C ABI in
// include/dsa_paged.h.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/dsa_paged.h"

namespace dsa_paged_k {

enum : int { ST_TIMEOUT = 1, ST_CHECK = 2 };

constexpr int kMaxGrid = 1024;  // CTAs of the attention at most
constexpr int kCounters = 2 * kMaxGrid;  // one per CTA and softmax group

constexpr int kEMin = -72, kEMax = 120;  // exponents of the append's scales

constexpr int kMaxLen = 0x7fffff00;  // tokens of a sequence at most: positions rounded up to a tile stay in 31 bits

// The batch of a call (device memory) and what bounds it.
struct Batch {
    const int32_t *cu, *lens, *table;
    int n_seqs, n_tokens, width;
    int page_log2, num_pages;
    int *status;
};

// Sequence s: rows row .. row + n - 1 are its new tokens, len its length with
// them.  One that does not fit the batch has no new tokens (and is reported
// by the caller: `bad`).
struct Seq {
    int row, n, len;
    bool bad;
};

__device__ __forceinline__ Seq make_seq(const Batch &b, int c0, int c1, int len)
{
    Seq q;
    q.row = c0;
    q.n = c1 - c0;
    q.len = len;
    q.bad = c0 < 0 || c1 < c0 || c1 > b.n_tokens || len < q.n || len > kMaxLen ||
            (long long)len > ((long long)b.width << b.page_log2);
    if (q.bad) q.n = 0;
    return q;
}

__device__ __forceinline__ Seq load_seq(const Batch &b, int s)
{
    return make_seq(b, __ldg(b.cu + s), __ldg(b.cu + s + 1), __ldg(b.lens + s));
}

}  // namespace dsa_paged_k

struct dsa_paged_ctx {
    uint32_t magic;
    int device, sms;
    int Hq, Hk, D, page, page_log2, num_pages, dtype;
    void *pages;
    float *scales;
    int *status;
    float *work;        // pieces of sequences shared by several CTAs
    int *counters;
    int grid[5];        // CTAs of each row block's kernel
    CUtensorMap map;    // the pool as rows of [K | V] in columns of 128 bytes
    uint32_t wait_limit;
};

namespace dsa_detail {
// The attention's side of dsa_paged_create (its workspace and tensor map)
// and its launch (dsa_paged_attn.cu); arguments are checked by the caller.
__attribute__((visibility("hidden"))) int paged_attn_init(dsa_paged_ctx *h);
__attribute__((visibility("hidden"))) int paged_attn_launch(dsa_paged_ctx *h, const dsa_paged_k::Batch &b, int max_new,
                                                            const void *q, void *out, cudaStream_t st);
}  // namespace dsa_detail
