// dsa_paged.cu -- the paged KV cache: its handle, and appending keys and
// values (bf16, or E4M3 with one scale per page, head and K / V) with the
// position rotation on the way.  C ABI in include/dsa_paged.h.
//
// The append reads q, k and v once and writes q, the pages and a scale per
// page, head and K / V: HBM bounds it, and latency for single tokens.  Its
// unit is a chunk, the new tokens of one sequence that fall into one page:
// a scale needs them all, and no two chunks share a page.  CTA (c, y) takes
// heads of part y of chunk c.  For E4M3 it first reads k and v for their
// largest values (they are in L1 or L2 the second time), grows the scales
// and re-rounds the codes already in the page where one grew; then, 16
// tokens at a time, it fills a table of sines in shared memory and rotates,
// codes and stores.  A row is covered by D / 16 threads with 8 elements of
// each half, so that the rotation needs no exchange.
//
// Measured (called): 8 prompts, 8200 tokens of 32 + 2 * 8 heads of 128, into
// E4M3 35.5 us (153 MB, 0.64 of the copy bandwidth: 47% of the issue slots go to
// scales, sines and codes, the rest waits for loads, two CTAs an SM); 7 prompts
// into bf16, 24 + 2 * 8 heads of 64, 13.6 us (46 MB, 0.5); 96 single tokens 5.4 us
// replayed from a graph (4.4 in bf16), a chain of dependent loads (length, page,
// scale, rows).
#include <cuda_fp8.h>

#include <climits>
#include <new>

#include "dsa_internal.h"
#include "dsa_paged.cuh"
#include "dsa_ptx.cuh"
#include "dsa_rope.cuh"

namespace dsa_paged_k {

using namespace dsa;

constexpr int kAppendThreads = 256;
constexpr int kRun = 16;        // tokens whose sines are in shared memory at once
constexpr int kMaxParts = 256;  // (head, K / V) pairs whose scales one CTA holds

struct AppendParams {
    Batch b;
    int chunk_log2;   // tokens of a chunk at most
    const int32_t *pos;
    const __nv_bfloat16 *q, *k, *v;
    long long qs, ks, vs;
    __nv_bfloat16 *q_out;
    void *pages;
    float *scales;
    int Hq, Hk;       // Hq 0: no queries
    RopeTable rope;   // pairs 0: no rotation
};

// The smallest e with a <= 448 * 2^e (a = 1.75 * 2^8 at e = 0).
__device__ __forceinline__ int exponent_v(float a)
{
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
    return min(max(e, kEMin), kEMax);
}

// The smallest e with a <= (448 * 2^e)^2 (a = 1.53125 * 2^17 at e = 0).  Below
// 2^-126 a mantissa has no leading one; both candidates are known there.
__device__ __forceinline__ int exponent_k(float a)
{
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - 17 + ((u & 0x7fffffu) > 0x440000u);
    return a < 0x1p-126f ? kEMin + (a > 0x1.88p-127f) : min(max((e + 1) >> 1, kEMin), kEMax);
}

__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float finite_or_0(float x) { return fabsf(x) <= 3.402823466e38f ? x : 0.f; }

// 8 E4M3 codes of v[i] * inv (nearest even, saturating, NaN kept).
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv)
{
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// 8 codes times `ratio`, as codes again.
__device__ __forceinline__ uint2 recode8(uint2 x, float ratio)
{
    const uint32_t w[2] = {x.x, x.y};
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> 16 * (i & 1)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
    return codes8(v, ratio);
}

// Finds chunk c of the batch: its sequence, the position of its first token
// and the first of the next page (or the length).  All threads of the CTA
// call it; false past the last chunk.  CTAs of chunk 0 look at the whole
// batch, so that every sequence that does not fit is reported.
struct Chunk {
    int seq, row, first, end;
};

__device__ bool find_chunk(const Batch &b, int chunk_log2, int c, Chunk *found, int *warp_sum)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    bool here = false;
    for (int s0 = 0; s0 < b.n_seqs; s0 += kAppendThreads) {
        const int s = s0 + tid;
        Seq q = {0, 0, 0, false};
        if (s < b.n_seqs) q = load_seq(b, s);
        if (q.bad) atomicOr(b.status, ST_CHECK);
        const int p0 = (q.len - q.n) >> chunk_log2;
        const int mine = q.n > 0 ? ((q.len - 1) >> chunk_log2) - p0 + 1 : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int total = 0;
        for (int w = 0; w < kAppendThreads / 32; ++w) {
            if (w < warp) incl += warp_sum[w];
            total += warp_sum[w];
        }
        const int at = c - base - (incl - mine);
        if (at >= 0 && at < mine) {
            const int p = p0 + at;
            found->seq = s;
            found->first = max(q.len - q.n, p << chunk_log2);
            found->end = min(q.len, (p + 1) << chunk_log2);
            found->row = q.row + found->first - (q.len - q.n);
        }
        base += total;
        __syncthreads();
        here = c < base;
        if (here && c > 0) break;
    }
    return here;
}

// The largest value of a raw row half-pair that sets a scale: |v|, or for keys
// the squared norm of a rotated pair (square of another element) times unit^2.
__device__ __forceinline__ float reach8(const uint4 &lo, const uint4 &hi, bool value, int j0, int pairs, float unit)
{
    float a[8], b[8], top = 0.f;
    unpack8(lo, a);
    unpack8(hi, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = finite_or_0(a[i]) * unit, z = finite_or_0(b[i]) * unit;
        if (value)
            top = fmaxf(top, fmaxf(fabsf(x), fabsf(z)));
        else if (j0 + i < pairs)
            top = fmaxf(top, fmaf(x, x, z * z));  // z * z is exact: one rounding
        else
            top = fmaxf(top, fmaxf(x * x, z * z));
    }
    return top;
}

template <bool FP8, int D>
__global__ void __launch_bounds__(kAppendThreads, FP8 ? 3 : 4) append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int L = D / 16;                    // threads of a row
    constexpr int kRows = kAppendThreads / L;    // rows in hand at once
    constexpr int kBatch = 2;                    // rows whose loads a thread has in flight (3: 37 us, 4: 41, 2: 35 for 8.2 k tokens)
    constexpr int kKeep = kRun * L / 32;         // raw rows a thread keeps: a run of tokens over the lanes of a warp
    __shared__ __align__(16) float2 tab[kRun][D / 2];
    __shared__ float inv_scale[kMaxParts];
    __shared__ Chunk ch;
    __shared__ int warp_sum[kAppendThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    if (!find_chunk(p.b, p.chunk_log2, blockIdx.x, &ch, warp_sum)) return;

    const int m = ch.end - ch.first;                       // tokens of the chunk
    const int slot0 = ch.first & ((1 << p.b.page_log2) - 1);
    const int page = __ldg(p.b.table + (size_t)ch.seq * p.b.width + (ch.first >> p.b.page_log2));

    // Heads of this part: of queries, and of (KV head, K / V) pairs.
    const int Y = gridDim.y, y = blockIdx.y;
    const int q0 = p.Hq * y / Y, q1 = p.Hq * (y + 1) / Y;
    const int u0 = 2 * p.Hk * y / Y, u1 = 2 * p.Hk * (y + 1) / Y;
    const int r = threadIdx.x / L, j0 = threadIdx.x % L * 8;
    const size_t row_bytes = 2 * D * (FP8 ? 1 : 2);  // K and V of one token
    const int pairs = p.rope.pairs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    // Where the K (u even) or V (u odd) row of slot t of KV head u / 2 lies.
    auto stored = [&](int u, int t) {
        return static_cast<unsigned char *>(p.pages) +
               ((((size_t)page * p.Hk + (u >> 1)) << p.b.page_log2) + t) * row_bytes + (u & 1) * (row_bytes / 2);
    };
    auto given = [&](int u, int t) {
        return ((u & 1) ? p.v + (size_t)(ch.row + t) * p.vs : p.k + (size_t)(ch.row + t) * p.ks) + (size_t)(u >> 1) * D + j0;
    };
    auto raw = [](const __nv_bfloat16 *at) { return *reinterpret_cast<const uint4 *>(at); };
    // Fills the table of sines for tokens t0 .. t0 + mt - 1.
    auto fill = [&](int t0, int mt) {
        for (int i = threadIdx.x; i < mt * (D / 2); i += kAppendThreads) {
            const int t = i / (D / 2), j = i % (D / 2);
            if (j < pairs) tab[t][j] = rope_cos_sin(p.rope, j, p.pos + (size_t)(ch.row + t0 + t) * p.rope.axes);
        }
    };
    auto turn = [&](float (&a)[8], float (&b)[8], int t) {
        float2 cs[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float4 x = *reinterpret_cast<const float4 *>(&tab[t][j0 + e]);
            cs[e] = make_float2(x.x, x.y);
            cs[e + 1] = make_float2(x.z, x.w);
        }
        turn8(a, b, cs, j0, pairs);
    };

    // E4M3: a warp takes a part's tokens side by side where there are
    // several, several parts where the chunk is a token or three.  Rows of a
    // chunk of up to kRun tokens stay in registers between the search for the
    // largest value and the coding.
    constexpr int kSub = 32 / L;
    const int side = m >= kSub ? kSub : 1;
    const int per = kSub / side;             // parts of a warp
    const int sub = lane / L;
    const bool kept = FP8 && m <= side * kKeep;
    const int u_first = u0 + warp * per + sub / side;
    uint4 lo[FP8 ? kKeep : 1], hi[FP8 ? kKeep : 1];
    auto fetch = [&](int u) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int t = sub % side + i * side;
            if (u < u1 && t < m) {
                lo[i] = raw(given(u, t));
                hi[i] = raw(given(u, t) + D / 2);
            }
        }
    };
    if (kept) fetch(u_first);  // in flight while the sines are made
    fill(0, min(kRun, m));
    __syncthreads();
    const bool held = page >= 0 && page < p.b.num_pages;
    if (!held && threadIdx.x == 0) atomicOr(p.b.status, ST_CHECK);

    if (FP8 && held) {
        for (int u = u0 + warp * per; u < u1; u += kAppendThreads / 32 * per) {
            const int mine = u + sub / side;
            const bool value = mine & 1;
            float *const at = p.scales + (size_t)page * 2 * p.Hk + mine;
            const float old = mine < u1 && slot0 > 0 ? *at : 0.f;
            if (kept && u != u0 + warp * per) fetch(mine);
            auto search = [&](float unit) {
                float top = 0.f;
                if (kept) {
#pragma unroll
                    for (int i = 0; i < kKeep; ++i)
                        if (mine < u1 && sub % side + i * side < m) top = fmaxf(top, reach8(lo[i], hi[i], value, j0, pairs, unit));
                } else if (mine < u1) {
#pragma unroll 4
                    for (int t = sub % side; t < m; t += side)
                        top = fmaxf(top, reach8(raw(given(mine, t)), raw(given(mine, t) + D / 2), value, j0, pairs, unit));
                }
                for (int o = 1; o < L * side; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                return top;
            };
            const float top = search(1.f);
            int e = value ? exponent_v(top) : exponent_k(top);
            // A norm from 2^64 on: its square has left fp32.
            const bool beyond = !value && top == INFINITY;
            if (__any_sync(0xffffffffu, beyond)) {
                const int far = exponent_k(search(0x1p-66f)) + 66;
                if (beyond) e = min(far, kEMax);
            }
            __syncwarp();  // every lane has read the old scale
            if (mine < u1) {
                float scale = two_to(e);
                if (old >= scale) {
                    scale = old;
                } else if (slot0 > 0) {
                    for (int t = sub % side; t < slot0; t += side) {
                        uint2 *l = reinterpret_cast<uint2 *>(stored(mine, t) + j0);
                        uint2 *h = reinterpret_cast<uint2 *>(stored(mine, t) + j0 + D / 2);
                        *l = recode8(*l, old / scale);
                        *h = recode8(*h, old / scale);
                    }
                }
                if (lane % (L * side) == 0 && scale != old) *at = scale;
                const float inv = 1.f / scale;
                if (kept) {
#pragma unroll
                    for (int i = 0; i < kKeep; ++i) {
                        const int t = sub % side + i * side;
                        if (t < m) {
                            float a[8], b[8];
                            unpack8(lo[i], a);
                            unpack8(hi[i], b);
                            if (!value) turn(a, b, t);
                            *reinterpret_cast<uint2 *>(stored(mine, slot0 + t) + j0) = codes8(a, inv);
                            *reinterpret_cast<uint2 *>(stored(mine, slot0 + t) + j0 + D / 2) = codes8(b, inv);
                        }
                    }
                } else if (lane % (L * side) == 0) {
                    inv_scale[mine - u0] = inv;
                }
            }
            __syncwarp();
        }
    }
    if (FP8 && !kept) __syncthreads();

    for (int t0 = 0; t0 < m; t0 += kRun) {
        const int mt = min(kRun, m - t0);
        if (t0 > 0) {
            __syncthreads();
            fill(t0, mt);
            __syncthreads();
        }
        // Rows of (token, head), tokens outermost, a few rows' loads ahead of
        // their stores (q_out may be q): queries first, then K and V.
        const int nq = q1 - q0, nu = held && !kept ? u1 - u0 : 0;
        const float per_q = 1.f / nq, per_u = 1.f / nu;
        for (int i0 = r; i0 < mt * nq; i0 += kBatch * kRows) {
            uint4 x[kBatch], z[kBatch];
            int t[kBatch], h[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * kRows;
                t[k] = (int)((i + 0.5f) * per_q);  // i / nq
                h[k] = q0 + i - t[k] * nq;
                if (i < mt * nq) {
                    const __nv_bfloat16 *at = p.q + (size_t)(ch.row + t0 + t[k]) * p.qs + (size_t)h[k] * D + j0;
                    x[k] = raw(at);
                    z[k] = raw(at + D / 2);
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (i0 + k * kRows < mt * nq) {
                    __nv_bfloat16 *o = p.q_out + ((size_t)(ch.row + t0 + t[k]) * p.Hq + h[k]) * D + j0;
                    float a[8], b[8];
                    unpack8(x[k], a);
                    unpack8(z[k], b);
                    turn(a, b, t[k]);
                    store8(o, a);
                    store8(o + D / 2, b);
                }
            }
        }
        for (int i0 = r; i0 < mt * nu; i0 += kBatch * kRows) {
            uint4 x[kBatch], z[kBatch];
            int t[kBatch], u[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * kRows;
                t[k] = (int)((i + 0.5f) * per_u);
                u[k] = u0 + i - t[k] * nu;
                if (i < mt * nu) {
                    x[k] = raw(given(u[k], t0 + t[k]));
                    z[k] = raw(given(u[k], t0 + t[k]) + D / 2);
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (i0 + k * kRows < mt * nu) {
                    float a[8], b[8];
                    unpack8(x[k], a);
                    unpack8(z[k], b);
                    if (!(u[k] & 1)) turn(a, b, t[k]);
                    unsigned char *o = stored(u[k], slot0 + t0 + t[k]);
                    if (FP8) {
                        const float inv = inv_scale[u[k] - u0];
                        *reinterpret_cast<uint2 *>(o + j0) = codes8(a, inv);
                        *reinterpret_cast<uint2 *>(o + j0 + D / 2) = codes8(b, inv);
                    } else {
                        store8(reinterpret_cast<__nv_bfloat16 *>(o) + j0, a);
                        store8(reinterpret_cast<__nv_bfloat16 *>(o) + j0 + D / 2, b);
                    }
                }
            }
        }
    }
}

// Resets the error that the host has read and no other: one of the other kind,
// or of a call on another stream, is still to be read.
__global__ void clear_status(int *status, int bit) { atomicAnd(status, ~bit); }

}  // namespace dsa_paged_k

using dsa_detail::cuda_fail;
using dsa_detail::dev_alloc;
using dsa_detail::fail;

namespace {

constexpr uint32_t kPagedMagic = 0x44535047u;  // "DSPG"

bool valid(const dsa_paged_ctx *h) { return h != nullptr && h->magic == kPagedMagic; }

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

void free_paged(dsa_paged_ctx *h)
{
    if (!h) return;
    cudaFree(h->status);
    cudaFree(h->work);
    cudaFree(h->counters);
    h->magic = 0;
    delete h;
}

// Checks what append and attend share and fills the batch.
int make_batch(dsa_paged_ctx *h, int n_seqs, int n_tokens, const int32_t *cu, const int32_t *lens, const int32_t *table,
               int width, dsa_paged_k::Batch *b)
{
    if (n_seqs < 0 || n_tokens < 0 || width < 0)
        return fail(DSA_ERR_ARG, "n_seqs, n_tokens and table_width must be >= 0 (got %d, %d, %d)", n_seqs, n_tokens, width);
    if (n_seqs == INT_MAX) return fail(DSA_ERR_ARG, "n_seqs too large");
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    if (dev != h->device) return fail(DSA_ERR_ARG, "the handle was made on device %d, the current one is %d", h->device, dev);
    if (n_seqs > 0 && n_tokens > 0) {
        if (!cu || !lens || !table) return fail(DSA_ERR_ARG, "cu, lens and table must be non-NULL");
        if (((uintptr_t)cu | (uintptr_t)lens | (uintptr_t)table) % 4)
            return fail(DSA_ERR_ARG, "cu, lens and table must be 4-byte aligned");
    }
    b->cu = cu;
    b->lens = lens;
    b->table = table;
    b->n_seqs = n_seqs;
    b->n_tokens = n_tokens;
    b->width = width;
    b->page_log2 = h->page_log2;
    b->num_pages = h->num_pages;
    b->status = h->status;
    return DSA_OK;
}

// Memory of the device that the handle is made on: a kernel launched there
// would follow a pointer of another device, or of the host, all the same.
int check_memory(const char *name, const void *p, int device)
{
    cudaPointerAttributes a;
    cudaError_t e = cudaPointerGetAttributes(&a, p);
    if (e != cudaSuccess) return cuda_fail(e, "pointer query");
    if (a.type == cudaMemoryTypeManaged || (a.type == cudaMemoryTypeDevice && a.device == device)) return DSA_OK;
    if (a.type == cudaMemoryTypeDevice)
        return fail(DSA_ERR_ARG, "%s lie on device %d, the current one is %d", name, a.device, device);
    return fail(DSA_ERR_ARG, "%s must be device memory", name);
}

int check_stride(const char *name, int64_t stride, int64_t row)
{
    if (stride < row || stride % 8 || stride > LLONG_MAX / 16 / INT_MAX)
        return fail(DSA_ERR_ARG, "%s must be a multiple of 8 and at least one row, %lld (got %lld)", name, (long long)row,
                    (long long)stride);
    return DSA_OK;
}

}  // namespace

extern "C" {

int dsa_paged_create(int q_heads, int kv_heads, int head_dim, int page_size, int num_pages, int dtype, void *pages,
                     float *scales, dsa_paged *out)
{
    if (!out) return fail(DSA_ERR_ARG, "out is NULL");
    *out = nullptr;
    if (kv_heads < 1 || kv_heads > 1024) return fail(DSA_ERR_ARG, "kv_heads must be in [1, 1024] (got %d)", kv_heads);
    if (q_heads < 1 || q_heads > 65536 || q_heads % kv_heads)
        return fail(DSA_ERR_ARG, "q_heads must be a multiple of kv_heads up to 65536 (got %d and %d)", q_heads, kv_heads);
    if (head_dim != 64 && head_dim != 128) return fail(DSA_ERR_ARG, "head_dim must be 64 or 128 (got %d)", head_dim);
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return fail(DSA_ERR_ARG, "page_size must be 16, 32, 64 or 128 (got %d)", page_size);
    if (num_pages < 1 || (long long)num_pages * kv_heads * page_size > INT_MAX)
        return fail(DSA_ERR_ARG, "num_pages must be >= 1 and num_pages * kv_heads * page_size below 2^31 (got %d)", num_pages);
    if (dtype != DSA_BF16 && dtype != DSA_FP8_E4M3)
        return fail(DSA_ERR_ARG, "dtype must be DSA_BF16 or DSA_FP8_E4M3 (got %d)", dtype);
    if (!pages || (uintptr_t)pages % 128) return fail(DSA_ERR_ARG, "pages must be non-NULL and 128-byte aligned");
    if (dtype == DSA_FP8_E4M3 && (!scales || !aligned16(scales)))
        return fail(DSA_ERR_ARG, "scales must be non-NULL and 16-byte aligned for DSA_FP8_E4M3");
    if (dtype == DSA_BF16 && scales) return fail(DSA_ERR_ARG, "scales must be NULL for DSA_BF16");

    dsa_paged_ctx *h = new (std::nothrow) dsa_paged_ctx();
    if (!h) return fail(DSA_ERR_OOM, "host allocation failed");
    h->magic = kPagedMagic;
    h->Hq = q_heads;
    h->Hk = kv_heads;
    h->D = head_dim;
    h->page = page_size;
    h->page_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    h->num_pages = num_pages;
    h->dtype = dtype;
    h->pages = pages;
    h->scales = scales;
    h->wait_limit = 0xffffffffu;
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
    if (e != cudaSuccess) {
        free_paged(h);
        return cuda_fail(e, "device query");
    }
    int rc = check_memory("pages", pages, h->device);
    if (rc == DSA_OK && scales) rc = check_memory("scales", scales, h->device);
    if (rc == DSA_OK) rc = dev_alloc((void **)&h->status, 16, "paged cache status");
    if (rc == DSA_OK && (e = cudaMemset(h->status, 0, 16)) != cudaSuccess) rc = cuda_fail(e, "cudaMemset");
    if (rc == DSA_OK) rc = dsa_detail::paged_attn_init(h);
    if (rc != DSA_OK) {
        free_paged(h);
        return rc;
    }
    *out = h;
    return DSA_OK;
}

int dsa_paged_destroy(dsa_paged h)
{
    if (!h) return DSA_OK;
    if (!valid(h)) return fail(DSA_ERR_STATE, "invalid paged cache handle");
    cudaDeviceSynchronize();
    free_paged(h);
    return DSA_OK;
}

int dsa_paged_append(dsa_paged h, int n_seqs, int n_tokens, const int32_t *cu, const int32_t *lens,
                     const int32_t *table, int table_width, dsa_rope rope, const int32_t *pos, const void *q,
                     int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *q_out,
                     void *stream)
{
    if (!valid(h)) return fail(DSA_ERR_STATE, "invalid paged cache handle");
    dsa_paged_k::AppendParams p;
    int rc = make_batch(h, n_seqs, n_tokens, cu, lens, table, table_width, &p.b);
    if (rc != DSA_OK) return rc;
    p.rope.pairs = 0;
    if (rope) {
        int D = 0;
        const dsa::RopeTable *t = dsa_detail::rope_table(rope, &D);
        if (!t) return fail(DSA_ERR_STATE, "invalid rotation plan");
        if (D != h->D) return fail(DSA_ERR_ARG, "the plan's head_dim is %d, the cache's %d", D, h->D);
        p.rope = *t;
    }
    if (!rope != !pos && n_tokens > 0) return fail(DSA_ERR_ARG, "rope and pos go together");
    if (!q != !q_out && n_tokens > 0) return fail(DSA_ERR_ARG, "q and q_out go together");
    if (q && (rc = check_stride("q_stride", q_stride, (int64_t)h->Hq * h->D)) != DSA_OK) return rc;
    if ((rc = check_stride("k_stride", k_stride, (int64_t)h->Hk * h->D)) != DSA_OK) return rc;
    if ((rc = check_stride("v_stride", v_stride, (int64_t)h->Hk * h->D)) != DSA_OK) return rc;
    if (n_seqs == 0 || n_tokens == 0) return DSA_OK;
    if (!k || !v) return fail(DSA_ERR_ARG, "k and v must be non-NULL");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || (uintptr_t)pos % 4)
        return fail(DSA_ERR_ARG, "q, k, v and q_out must be 16-byte aligned, pos 4-byte aligned");
    if (q && q == q_out && q_stride != (int64_t)h->Hq * h->D)
        return fail(DSA_ERR_ARG, "in place, q must be contiguous (q_out is)");
    p.pos = pos;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.qs = q_stride;
    p.ks = k_stride;
    p.vs = v_stride;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.pages = h->pages;
    p.scales = h->scales;
    p.Hq = q ? h->Hq : 0;
    p.Hk = h->Hk;

    // Chunks: at most one per token, and per sequence at most one more than
    // full pages and the two ragged ends.  Heads are split over grid.y until
    // there are two CTAs an SM, in parts of 8 units at least, and so that a CTA
    // holds the scales of its parts.  With four asked for instead of two (graph
    // replays), E4M3: 96 single tokens 9.3 us instead of 5.5, 8 prompts of 1025
    // tokens 47 instead of 54, 8.2 k ragged prompt tokens 38 instead of 35; bf16:
    // 96 single tokens 6.7 instead of 4.4, 8 x 1025 tokens 46 instead of 41, one
    // prompt of 2048 20.5 instead of 16.8, 7 x 700 tokens with heads of 64 13.2
    // instead of 16.2.
    p.chunk_log2 = h->dtype == DSA_FP8_E4M3 ? h->page_log2 : 4;
    const long long bound = ((long long)n_tokens >> p.chunk_log2) + 2LL * n_seqs;
    const long long chunks = n_tokens < bound ? n_tokens : bound;
    const int units = p.Hq + 2 * p.Hk;
    long long Y = (2LL * h->sms + chunks - 1) / chunks;
    const long long most = (units + 7) / 8, least = (2 * p.Hk + dsa_paged_k::kMaxParts - 1) / dsa_paged_k::kMaxParts;
    if (Y > most) Y = most;
    if (Y < least) Y = least;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)chunks, (unsigned)Y);
    cfg.blockDim = dim3(dsa_paged_k::kAppendThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (h->dtype == DSA_FP8_E4M3)
        e = h->D == 128 ? cudaLaunchKernelEx(&cfg, dsa_paged_k::append_kernel<true, 128>, p)
                        : cudaLaunchKernelEx(&cfg, dsa_paged_k::append_kernel<true, 64>, p);
    else
        e = h->D == 128 ? cudaLaunchKernelEx(&cfg, dsa_paged_k::append_kernel<false, 128>, p)
                        : cudaLaunchKernelEx(&cfg, dsa_paged_k::append_kernel<false, 64>, p);
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "append launch");
}

int dsa_paged_attend(dsa_paged h, int n_seqs, int n_tokens, int max_new, const int32_t *cu, const int32_t *lens,
                     const int32_t *table, int table_width, const void *q, void *out, void *stream)
{
    if (!valid(h)) return fail(DSA_ERR_STATE, "invalid paged cache handle");
    dsa_paged_k::Batch b;
    int rc = make_batch(h, n_seqs, n_tokens, cu, lens, table, table_width, &b);
    if (rc != DSA_OK) return rc;
    if (max_new < 1) return fail(DSA_ERR_ARG, "max_new must be >= 1 (got %d)", max_new);
    if ((long long)n_tokens * h->Hq > INT_MAX)
        return fail(DSA_ERR_ARG, "n_tokens * q_heads must be below 2^31 (got %d x %d)", n_tokens, h->Hq);
    if (n_seqs == 0 || n_tokens == 0) return DSA_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out))
        return fail(DSA_ERR_ARG, "q and out must be non-NULL and 16-byte aligned");
    return dsa_detail::paged_attn_launch(h, b, max_new, q, out, (cudaStream_t)stream);
}

int dsa_paged_sync_status(dsa_paged h, void *stream)
{
    if (!valid(h)) return fail(DSA_ERR_STATE, "invalid paged cache handle");
    cudaStream_t st = (cudaStream_t)stream;
    int word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, h->status, 4, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e, "status copy");
    if (word == 0) return DSA_OK;
    const int bit = word & dsa_paged_k::ST_TIMEOUT ? dsa_paged_k::ST_TIMEOUT : dsa_paged_k::ST_CHECK;
    dsa_paged_k::clear_status<<<1, 1, 0, st>>>(h->status, bit);
    if ((e = cudaGetLastError()) != cudaSuccess || (e = cudaStreamSynchronize(st)) != cudaSuccess)
        return cuda_fail(e, "status reset");
    if (bit == dsa_paged_k::ST_TIMEOUT) return fail(DSA_ERR_TIMEOUT, "a bounded wait in the paged attention gave up");
    return fail(DSA_ERR_DEVICE_CHECK, "a sequence of the batch does not fit it, or a page number lies outside the pool");
}

int dsa_paged_set_wait_limit(dsa_paged h, uint32_t limit)
{
    if (!valid(h)) return fail(DSA_ERR_STATE, "invalid paged cache handle");
    h->wait_limit = limit;
    return DSA_OK;
}

}  // extern "C"
