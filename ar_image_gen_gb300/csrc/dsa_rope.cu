// dsa_rope.cu -- rotary position embedding with several position axes.  C ABI
// in include/dsa_rope.h.
//
// The rotation reads and writes every element once (6 flops a pair): HBM is
// the bound, and a launch's latency where there are few tokens.  A token's
// sines and cosines are shared by its heads, so a CTA takes whole tokens: its
// threads first fill a table of the tokens' pairs in shared memory, then each
// keeps 8 pairs of one token in registers and walks over heads, 16 bytes from
// the lower and 16 from the upper half of a head at a time.
//
// Measured: 8100 tokens x 64 heads of 128 in bf16 44.5 us (265 MB, 0.88 of the
// copy bandwidth); 4161 x 40 heads of 128 in fp32, 33.9 us (170 MB, 0.74); 32 tokens
// 2.6 us, a launch's latency.
#include <cmath>
#include <climits>
#include <new>

#include "../../include/dsa.h"
#include "../../include/dsa_rope.h"
#include "dsa_internal.h"
#include "dsa_ptx.cuh"
#include "dsa_rope.cuh"

namespace dsa_rope_k {

using namespace dsa;

constexpr int kThreads = 256;
constexpr int kGroups = 8;  // of threads that share a token, at least

struct Params {
    const int32_t *pos;
    const void *x;
    void *y;
    long long xs, ys;
    int tokens, heads;
    int groups;  // threads of one token that share its 8-pair runs, each with heads g, g + groups, ..
    float sign;
    RopeTable rope;
};

// CTAs an SM: with 3 asked for, fp32 took 34.8 us instead of 33.9 (its loads in
// flight wait for registers); with 2, bf16 45.5 us instead of 44.5.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 4) rope_kernel(const __grid_constant__ Params p)
{
    constexpr int L = D / 16;  // threads that cover one head
    __shared__ float2 tab[kThreads / (L * kGroups)][D / 2];
    pdl_wait();
    pdl_launch_dependents();
    const int per = L * p.groups, nt = kThreads / per;  // threads of a token, tokens of this CTA
    const int n0 = blockIdx.x * nt;
    for (int i = threadIdx.x; i < nt * (D / 2); i += kThreads) {
        const int n = i / (D / 2), j = i % (D / 2);
        if (n0 + n < p.tokens && j < p.rope.pairs) {
            float2 cs = rope_cos_sin(p.rope, j, p.pos + (size_t)(n0 + n) * p.rope.axes);
            cs.y *= p.sign;
            tab[n][j] = cs;
        }
    }
    __syncthreads();
    const int n = threadIdx.x / per, g = threadIdx.x % per / L, j0 = threadIdx.x % L * 8;
    if (n >= nt || n0 + n >= p.tokens) return;
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = tab[n][j0 + i];
    const T *x = static_cast<const T *>(p.x) + (size_t)(n0 + n) * p.xs + j0;
    T *y = static_cast<T *>(p.y) + (size_t)(n0 + n) * p.ys + j0;
    // Two heads at a time, loads first: x and y may be the same rows, so the
    // compiler cannot move a load above the store of the head before.
    for (int h = g; h < p.heads; h += 2 * p.groups) {
        Raw8<T> a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (h + i * p.groups < p.heads) {
                a[i].load(x + (size_t)(h + i * p.groups) * D);
                b[i].load(x + (size_t)(h + i * p.groups) * D + D / 2);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (h + i * p.groups < p.heads) {
                float u[8], w[8];
                a[i].get(u);
                b[i].get(w);
                turn8(u, w, cs, j0, p.rope.pairs);
                store8(y + (size_t)(h + i * p.groups) * D, u);
                store8(y + (size_t)(h + i * p.groups) * D + D / 2, w);
            }
        }
    }
}

}  // namespace dsa_rope_k

using dsa_detail::cuda_fail;
using dsa_detail::fail;

namespace {

constexpr uint32_t kRopeMagic = 0x44535252u;  // "DSRR"

// 2^64 f / (2 pi) modulo 2^64, the double f taken as exact: its mantissa
// times the first 128 binary digits of 1 / (2 pi).
uint64_t turns64(double f)
{
    int e;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(f, &e), 53);  // f = m 2^(e - 53), f <= 1 here
    const unsigned __int128 inv = ((unsigned __int128)0x28be60db9391054aull << 64) | 0x7f09d5f47d4d3770ull;
    // m * inv has up to 181 bits: the part above 2^64 and the part below
    const unsigned __int128 lo = (unsigned __int128)(uint64_t)inv * m, hi = (unsigned __int128)(uint64_t)(inv >> 64) * m;
    const unsigned __int128 top = hi + (lo >> 64);  // f / (2 pi) = top 2^(e - 53 - 64)
    const int s = 53 - e;                           // >= 52: shift that leaves 64 fraction bits
    return s >= 128 ? 0 : (uint64_t)(top >> s);
}

template <typename T>
cudaError_t launch(const dsa_rope_k::Params &p, int D, unsigned grid, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(dsa_rope_k::kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return D == 128 ? cudaLaunchKernelEx(&cfg, dsa_rope_k::rope_kernel<T, 128>, p)
                    : cudaLaunchKernelEx(&cfg, dsa_rope_k::rope_kernel<T, 64>, p);
}

}  // namespace

const dsa::RopeTable *dsa_detail::rope_table(const dsa_rope_ctx *r, int *head_dim)
{
    if (!r || r->magic != kRopeMagic) return nullptr;
    *head_dim = r->D;
    return &r->table;
}

extern "C" {

int dsa_rope_create(int head_dim, int axes, const int *pairs, int restart, double base, dsa_rope *out)
{
    if (!out) return fail(DSA_ERR_ARG, "out is NULL");
    *out = nullptr;
    if (head_dim != 64 && head_dim != 128) return fail(DSA_ERR_ARG, "head_dim must be 64 or 128 (got %d)", head_dim);
    if (axes < 1 || axes > 4) return fail(DSA_ERR_ARG, "axes must be in [1, 4] (got %d)", axes);
    if (!pairs) return fail(DSA_ERR_ARG, "pairs is NULL");
    if (!(base > 1.0) || !std::isfinite(base)) return fail(DSA_ERR_ARG, "base must be finite and above 1 (got %g)", base);
    int sum = 0;
    for (int a = 0; a < axes; ++a) {
        if (pairs[a] < 1 || pairs[a] > head_dim / 2)
            return fail(DSA_ERR_ARG, "axis %d must own 1 to %d pairs (got %d)", a, head_dim / 2, pairs[a]);
        sum += pairs[a];
    }
    if (sum > head_dim / 2)
        return fail(DSA_ERR_ARG, "the axes own %d pairs, a head has %d", sum, head_dim / 2);
    dsa_rope_ctx *r = new (std::nothrow) dsa_rope_ctx();
    if (!r) return fail(DSA_ERR_OOM, "host allocation failed");
    r->magic = kRopeMagic;
    r->D = head_dim;
    r->table.pairs = sum;
    r->table.axes = axes;
    for (int a = 0, j = 0; a < axes; ++a)
        for (int i = 0; i < pairs[a]; ++i, ++j) {
            r->table.axis[j] = (unsigned char)a;
            r->table.freq[j] = turns64(restart ? std::pow(base, -(double)i / pairs[a]) : std::pow(base, -2.0 * j / head_dim));
        }
    *out = r;
    return DSA_OK;
}

int dsa_rope_destroy(dsa_rope r)
{
    if (!r) return DSA_OK;
    if (r->magic != kRopeMagic) return fail(DSA_ERR_STATE, "invalid rotation plan");
    r->magic = 0;
    delete r;
    return DSA_OK;
}

int dsa_rope_apply(dsa_rope r, int tokens, int heads, int dtype, const int32_t *pos, const void *x, int64_t x_stride,
                   void *y, int64_t y_stride, int inverse, void *stream)
{
    int D = 0;
    const dsa::RopeTable *table = dsa_detail::rope_table(r, &D);
    if (!table) return fail(DSA_ERR_STATE, "invalid rotation plan");
    if (tokens < 0) return fail(DSA_ERR_ARG, "tokens must be >= 0 (got %d)", tokens);
    if (heads < 1 || heads > 65536) return fail(DSA_ERR_ARG, "heads must be in [1, 65536] (got %d)", heads);
    if (dtype != DSA_BF16 && dtype != DSA_F32) return fail(DSA_ERR_ARG, "dtype must be DSA_BF16 or DSA_F32 (got %d)", dtype);
    const int vec = dtype == DSA_BF16 ? 8 : 4;
    const int64_t row = (int64_t)heads * D;
    if (x_stride < row || y_stride < row || x_stride % vec || y_stride % vec)
        return fail(DSA_ERR_ARG, "strides must be at least heads * head_dim and multiples of 16 bytes (got %lld, %lld)",
                    (long long)x_stride, (long long)y_stride);
    if (x_stride > LLONG_MAX / 8 / ((int64_t)tokens + 1) || y_stride > LLONG_MAX / 8 / ((int64_t)tokens + 1))
        return fail(DSA_ERR_ARG, "stride too large");
    if (tokens == 0) return DSA_OK;
    if (!pos || !x || !y) return fail(DSA_ERR_ARG, "pos, x and y must be non-NULL");
    if ((uintptr_t)x % 16 || (uintptr_t)y % 16 || (uintptr_t)pos % 4)
        return fail(DSA_ERR_ARG, "x and y must be 16-byte aligned, pos 4-byte aligned");
    if (x == y && x_stride != y_stride) return fail(DSA_ERR_ARG, "in place, x and y have the same stride");

    dsa_rope_k::Params p;
    p.pos = pos;
    p.x = x;
    p.y = y;
    p.xs = x_stride;
    p.ys = y_stride;
    p.tokens = tokens;
    p.heads = heads;
    p.sign = inverse ? -1.f : 1.f;
    p.rope = *table;
    // A token's 8-pair runs are shared by `groups` threads: as many as there
    // are heads while the tokens do not fill the device, else kGroups, so that a
    // CTA's table of sines (one entry a thread) serves 8 heads a thread.
    const int L = D / 16;
    const int most = tokens <= 1024 ? dsa_rope_k::kThreads / L : dsa_rope_k::kGroups;
    p.groups = dsa_rope_k::kGroups;
    while (p.groups < most && p.groups < heads) p.groups *= 2;
    const int nt = dsa_rope_k::kThreads / (L * p.groups);
    const unsigned grid = (unsigned)((tokens + (long long)nt - 1) / nt);
    cudaError_t e = dtype == DSA_BF16 ? launch<__nv_bfloat16>(p, D, grid, (cudaStream_t)stream)
                                      : launch<float>(p, D, grid, (cudaStream_t)stream);
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "rotation launch");
}

}  // extern "C"
