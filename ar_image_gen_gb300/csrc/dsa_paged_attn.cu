// dsa_paged_attn.cu -- attention over the paged KV cache on the tensor cores.
// C ABI in include/dsa_paged.h.
//
// Two kernels, by the rows (new token x grouped query head) that a sequence
// has for one KV head.  The second, for blocks of 128 rows, is described where
// it begins.  The first computes, per tile of 128 keys and block of up to 32
// rows,
//
//     S^T = K Q^T          [128 keys x rows]      (tcgen05.mma, M = keys)
//     w   = 2^(S^T c - m)  softmax weights, m a running reference per row
//     O^T += V^T w         [head_dim x rows]      (tcgen05.mma, M = head_dim)
//
// so that both products take the cache's rows as the wide operand straight
// from shared memory, where TMA put them page by page (128-byte swizzle, K
// as the K-major, V as the M-major operand): no key or value passes through
// a register, and a handful of rows fills the 128-row tensor-core tile.
//
// An E4M3 cache is multiplied as E4M3, the other operand split into numbers of
// 8 bits in columns of their own (a tile has 16 at the least).  A bf16 query is
// t1 + t2 / 16 of two E4M3 numbers, exactly (8 = 4 + 4 significant bits) but for
// elements under 2^-22 of its row's largest.  A weight is the sum of three E5M2
// numbers: 9 bits, down to 2^-28 of the reference, so that thousands of keys
// beside a dominant one keep theirs.  (Two E4M3 numbers, 8 bits down to 2^-18,
// lost 90 % of an output that 8200 keys of e^-13 to e^-15 made up; they took 55.9
// us instead of 56.2 for 96 sequences of 65 to 640 keys, 85.9 instead of 88.5 for
// 32 x 4000 keys x 32 rows.)  The scale of a page and head enters the logit (K) and
// the weight (V); since a page's weight times its scale is what is rounded, m
// refers to logit + log2(V scale).
//
// Over a bf16 cache a weight is the sum of two bf16 numbers, to 2^-16 of it, in
// columns of their own likewise.  The second costs nothing where the cache's
// bytes are the bound: 16 sequences of 65 to 4160 keys take 89.0 us with one
// term, 89.5 with two.
//
// m grows only when a weight would pass 2^SLACK: then the four softmax warps
// agree on new references and rescale O in tensor memory.  Otherwise a tile
// costs them one barrier.
//
// Work: the tiles of all (sequence, row block, KV head) in order are divided
// evenly over a persistent grid; an item that several CTAs share is joined by
// the one that finishes last, in the order of the keys.  (Runs drawn from a
// counter instead took longer in every mix of lengths but one of equal short
// sequences: the draw and the search for its sequence cost more than the
// imbalance.)
//
// What bounds it: with few rows and many keys the bytes of the cache.  One new
// token of 16 sequences of 65 to 4160 keys, 32 heads of 128, bf16: 89 us called,
// 0.92 of the copy bandwidth.  96 sequences of 65 to 640 keys in E4M3: 56.4 us,
// 0.73, the rest being the items' beginnings and ends (32 heads a sequence, 3
// tiles each on average).  One sequence is bound by latency: 10.6 us at 607 keys,
// the launch, the division of the work and a head's 5 tiles one after another in
// one CTA (see kWhole).
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "dsa_decode.cuh"
#include "dsa_internal.h"
#include "dsa_paged.cuh"
#include "dsa_tc.cuh"

namespace dsa_paged_k {

using namespace dsa;

constexpr int kSoft = 128;     // threads of a softmax group: one per key of a tile
constexpr uint32_t kSoftBar = 1;  // named barrier of the first softmax group
constexpr int kTile = 128;     // keys of a tile
constexpr uint32_t kBox = kTile * 128;  // bytes of one 128-byte column of a tile
// Reference of a published row that no logit above -infinity has set, and of
// rows that a group has beyond its block: they weigh nothing and set none.
constexpr float kNoMax = -3.402823466e38f;
constexpr float kNever = 1e30f;
// Of an E4M3 cache the reference is log2 of the largest weight x V scale, less
// this.  A row's sum adds up the weights themselves, 2^kLow over the V scale of
// the page that set the reference: with scales of 2^-72 to 2^120 from 2^-102,
// where a key that weighs 2^-24 of it is still a normal number, to 2^96, which
// 2^31 keys do not carry out of fp32.  (From 0 instead, V of 1e36 lost the keys
// under 2^-7 of the largest.)
constexpr int kLow = 18;
constexpr uint32_t kBarBytes = 320;
constexpr int kScaleRing = 8;  // tiles whose page scales are in shared memory

struct AttnParams {
    Batch b;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    const float *scales;
    float *work;
    int *counters;
    int Hq, Hk, G;
    uint32_t g_mul;  // ceil(2^32 / G) where rows x G stay below 2^32, else 0
    uint32_t wait_limit;
    int lead;        // places of an item of 128 rows beside its tiles: its queries' bytes count

    // x / G for a row x of a sequence: the runtime's division by a variable is long, and the walks do it per block.
    __device__ __forceinline__ int over_g(int x) const { return g_mul ? (int)__umulhi((uint32_t)x, g_mul) : G == 1 ? x : x / G; }
};

// What the softmax and MMA warps need of an item (a row block of one sequence
// and KV head, and the part of its tiles in the CTA's run); written by the
// query warp.  t1 == 0: no further item.
struct Info {
    int nr;              // rows of the block
    int limit, least;    // keys that its last and its first row attend
    int t0, t1;          // tiles
    int more;            // another item follows
    int first, pieces;   // CTA of the item's first tile; CTAs that share the item
};

// Words of a CTA beside its items'.
struct Shared {
    uint32_t tmem;   // address of its tensor memory
    int last[2];     // of each group: its piece of the shared item came last
    int arrived[2];  // shared items whose counters the groups have added to
    int gave_up;     // a group has left items undone
    int pad[2];
};

template <bool FP8, int D, int RB>
struct Shape {
    static constexpr int EB = FP8 ? 1 : 2;
    // Groups of an MMA warp and 4 softmax warps, each with up to RW rows of the
    // block and columns of its own: they run out of step, so that one computes
    // while the other waits.
    static constexpr int GROUPS = RB == 32 ? 2 : 1;
    static constexpr int RW = RB / GROUPS;
    static constexpr int THREADS = 32 * (2 + 5 * GROUPS);  // and a producer and a query warp
    static constexpr int SOFT = 1 + GROUPS, QUERY = 1 + 5 * GROUPS;  // first softmax warp, query warp
    static constexpr int QD = RB == 2 ? 3 : 2;             // items whose queries are in shared memory
    static constexpr int TERMS = FP8 ? 2 : 1;    // numbers that a query's element is split into
    static constexpr int WTERMS = FP8 ? 3 : 2;   // and a weight
    static constexpr int NS = TERMS * RW < 16 ? 16 : TERMS * RW;    // columns of a group's S^T
    static constexpr int NO = (WTERMS * RW + 15) / 16 * 16;         // and O^T
    // A bf16 tile of head_dim 128 goes through the ring of slots as its K part
    // and its V part, others whole.  A part is C columns of 128 bytes; 8 keys of
    // column 0, the same keys of column 1, .., then the next 8 keys.
    static constexpr int PARTS = D * EB == 256 ? 2 : 1;
    static constexpr int C = 2 * D * EB / 128 / PARTS;
    static constexpr uint32_t SLOT = C * kBox;
    static constexpr uint32_t SBO = C * 1024;                    // from 8 keys to the next 8
    static constexpr uint32_t VCOL = !FP8 || D == 64 ? 0 : 1024; // first column of M in O^T (see the epilogue for 64)
    static constexpr int QBOXES = D * EB < 128 ? 1 : D * EB / 128;
    // Rows of a group's queries' and weights' operands that exist; the columns
    // past the terms of RW rows read whatever follows and are never looked at.
    static constexpr int QROWS = TERMS * RW < 8 ? 8 : TERMS * RW;
    static constexpr int PROWS = WTERMS * RW < 8 ? 8 : WTERMS * RW;
    static constexpr int PBOXES = kTile * EB / 128;
    static constexpr uint32_t QGROUP = QBOXES * QROWS * 128, PGROUP = PBOXES * PROWS * 128;
    static constexpr uint32_t QBUF = GROUPS * QGROUP, PBUF = GROUPS * PGROUP;
    static constexpr int GCOLS = 2 * (NS + NO);                  // of a group: S^T twice, O^T twice
    static constexpr int TCOLS = GCOLS * GROUPS;
    static constexpr int TMEM = TCOLS <= 64 ? 64 : TCOLS <= 128 ? 128 : TCOLS <= 256 ? 256 : 512;
    // log2 of how far a weight may pass 1 before the references move, and of
    // the factor that weights are held with (fp16 reaches 2^16, E5M2 almost).
    static constexpr int SLACK = FP8 ? 3 : 8;
    static constexpr int LOW = FP8 ? kLow : 0;
    static constexpr int HELD = FP8 ? 15 - SLACK - LOW : 0;
    static constexpr int PIECE = RB * (D + 2);  // floats of a published piece: O, m, l
    // Few rows leave the tensor cores idle while a tile's weights are made:
    // other CTAs of the SM fill in.  In bf16 a block of 16 takes one CTA with
    // 6 slots instead of two with 2: 32 sequences x 4000 keys, 64 heads over 4
    // of 64, 37.5 us and 39.4; 4 x 20000 keys 32.5 and 35.3.
    static constexpr int CTAS = RB <= 8 || (RB == 16 && FP8) ? 2 : 1;
    static constexpr uint32_t ROWF = (3 * QD + 8 + 8 + 2) * (RB < 8 ? 8 : RB);  // qc, bound, orow [QD], wmax, lsum [2][4], m [2]
    static constexpr uint32_t FIXED = QD * QBUF + 2 * PBUF + kBarBytes + kScaleRing * 64 + ROWF * 4 + QD * sizeof(Info) + sizeof(Shared) + 1024;
    static constexpr uint32_t ROOM = (228 * 1024) / CTAS - 1024 - 256;
    static constexpr int SLOTS = (ROOM - FIXED) / SLOT > 8 ? 8 : (ROOM - FIXED) / SLOT;
    static constexpr uint32_t OFF_Q = SLOTS * SLOT;
    static constexpr uint32_t OFF_P = OFF_Q + QD * QBUF;
    static constexpr uint32_t OFF_BAR = OFF_P + 2 * PBUF;
    static constexpr uint32_t OFF_SC = OFF_BAR + kBarBytes;      // [kScaleRing][8][2] page scales
    static constexpr uint32_t OFF_ROW = OFF_SC + kScaleRing * 64;
    static constexpr uint32_t OFF_INFO = OFF_ROW + ROWF * 4;
    static constexpr uint32_t SMEM = OFF_INFO + QD * sizeof(Info) + sizeof(Shared) + 1024;  // TMEM address, flags; alignment slack
    static_assert(SLOTS >= PARTS + 1 && (2 * SLOTS + 7 * GROUPS + 2 * QD) * 8 <= (int)kBarBytes, "slots of K and V");
    static_assert(SMEM <= ROOM && TCOLS <= TMEM && TMEM * CTAS <= 512, "shared and tensor memory of a CTA");
};

template <int RB>
__device__ __forceinline__ int block_limit(const Seq &q, const AttnParams &p, int rb)
{
    const int last = min((rb + 1) * RB, q.n * p.G) - 1;
    return q.len - q.n + p.over_g(last) + 1;
}

template <int RB>
__device__ __forceinline__ int block_tiles(const Seq &q, const AttnParams &p, int rb)
{
    return (block_limit<RB>(q, p, rb) + kTile - 1) / kTile;
}

// The places of a tile and of an item beside its tiles (its queries, first
// maximum and epilogue) on the cost line that is divided over the CTAs.  Up to
// 16 rows a tile costs its bytes; with 32, the weights of its rows, a softmax
// group's 8 at a time; with 128 rows as lanes, the same whatever they are.  The
// beginning of an item of 128 rows is head_dim / 16 tiles long: with 4 instead
// of 8 at 128, 2 prompts of 4096 tokens took 313 us instead of 276 (bf16), 616
// instead of 434 (E4M3), because the CTAs with the short items at a prompt's
// beginning came last; with 8 instead of 4 at 64, prompts of 2048 took 122 us
// instead of 116.
template <int RB>
__device__ __forceinline__ int tile_cost(int rows)
{
    return RB == 32 ? 2 + (rows + 15) / 16 : 1;
}
template <int RB>
__device__ __forceinline__ int item_lead(const AttnParams &p)
{
    return RB <= 16 ? 1 : RB == 128 ? p.lead : 12;
}
// An item of up to this many places, 640 keys of single tokens, is not split: it
// belongs to the run that holds its beginning.  A shared item's pieces are
// published, counted and joined, which takes longer than its tiles one after
// another, also where other CTAs are idle.  Whole and split (graph replays, 32
// heads over 32 or 8 of 128), keys 200, 300, 640: 1 sequence over 32 in bf16 7.7,
// 9.0, 9.5 us and 9.9, 10.4, 10.4; over 8 7.7, 8.7, 9.3 and 9.8, 10.0, 10.2; 8
// sequences over 32 9.1, 10.7, 11.2 and 14.6, 15.7, 14.6; in E4M3 8.1, 9.2, 9.7 and
// 13.8, 14.7, 13.4; 96 sequences in E4M3 41.8, 51.4, 80.8 and 44.6, 53.4, 82.6.
// Items of more places are the same in both.
template <int RB>
constexpr int kWhole = RB <= 16 ? 6 : 0;
template <int RB>
constexpr int kLeastRun = RB == 32 ? 8 : 1;  // places of a run at least: a tile begins in each

template <int RB>
__device__ __forceinline__ int block_rows(const Seq &q, int G, int rb)
{
    return min(RB, q.n * G - rb * RB);
}

// Places of one item of a row block, and of a sequence.
template <int RB>
__device__ __forceinline__ int item_cost(const Seq &q, const AttnParams &p, int rb)
{
    return block_tiles<RB>(q, p, rb) * tile_cost<RB>(block_rows<RB>(q, p.G, rb)) + item_lead<RB>(p);
}
template <int RB>
__device__ __forceinline__ long long seq_cost(const Seq &q, const AttnParams &p)
{
    long long t = 0;
    const int blocks = (int)(((long long)q.n * p.G + RB - 1) / RB);
    for (int rb = 0; rb < blocks; ++rb) t += item_cost<RB>(q, p, rb);
    return t * p.Hk;
}

// One (sequence, row block, KV head) and the part of its tiles in a run.
struct Item {
    int seq, row, n, len;
    int rb, head;
    int tiles, t0, t1, weight;
    long long x;         // place of its first tile
    __device__ __forceinline__ bool split() const { return t0 > 0 || t1 < tiles; }  // other CTAs have tiles of it
};

// Walks the items of a run [x0, x1) of the cost line: an item takes item_lead,
// then tile_cost for each tile, and a tile belongs to the run that holds its
// first place (those of an item that is not split, the item's).
template <int RB>
struct Walk {
    const AttnParams &p;
    long long x0, x1, at;  // at: where the next item begins
    int s, rb, head, blocks, tiles, weight;
    Seq q;

    __device__ __forceinline__ Walk(const AttnParams &p_, long long x0_, long long x1_, int s_, long long base)
        : p(p_), x0(x0_), x1(x1_), at(base), s(s_), head(0)
    {
        if (x0 >= x1) return;
        open();
        for (; rb + 1 < blocks; block(rb + 1)) {  // to the row block, then the head, that holds x0
            const long long span = (long long)(tiles * weight + item_lead<RB>(p)) * p.Hk;
            if (x0 < at + span) break;
            at += span;
        }
        head = (int)((x0 - at) / (tiles * weight + item_lead<RB>(p)));
        at += (long long)head * (tiles * weight + item_lead<RB>(p));
    }
    __device__ __forceinline__ void block(int i)
    {
        rb = i;
        tiles = block_tiles<RB>(q, p, i);
        weight = tile_cost<RB>(block_rows<RB>(q, p.G, i));
    }
    __device__ __forceinline__ void open()
    {
        q = load_seq(p.b, s);
        blocks = (int)(((long long)q.n * p.G + RB - 1) / RB);
        rb = 0;
        if (blocks > 0) block(0);
    }
    __device__ __forceinline__ bool next(Item &it)
    {
        while (at < x1) {
            if (head == p.Hk) {
                head = 0;
                if (++rb < blocks) block(rb);
            }
            if (rb >= blocks) {
                if (s + 1 >= p.b.n_seqs) return false;
                ++s;
                open();
                continue;
            }
            it.x = at + item_lead<RB>(p);
            if (tiles * weight + item_lead<RB>(p) <= kWhole<RB>) {
                it.t0 = 0;
                it.t1 = at >= x0 ? tiles : 0;
                at = it.x + tiles * weight;
            } else {
                it.t0 = x0 > it.x ? (int)((x0 - it.x + weight - 1) / weight) : 0;
                at = it.x + tiles * weight;
                it.t1 = x1 <= it.x ? 0 : x1 < at ? (int)((x1 - it.x + weight - 1) / weight) : tiles;
            }
            it.seq = s;
            it.row = q.row;
            it.n = q.n;
            it.len = q.len;
            it.rb = rb;
            it.head = head;
            it.tiles = tiles;
            it.weight = weight;
            ++head;
            if (it.t0 < it.t1) return true;
        }
        return false;
    }
};

// Bounded wait of a whole warp: all its lanes learn the same outcome and leave
// together, so what follows may need them converged.  A poll sleeps until the
// phase completes or about kPollHint nanoseconds pass; the timer is read only
// once a wait has become long.  Gives up after `limit` polls or about a second.
constexpr uint32_t kPollHint = 4000;

__device__ __forceinline__ bool wait_poll(uint32_t bar, uint32_t parity, uint32_t limit)
{
    uint32_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 0; i < limit; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, kPollHint))) return true;
        if ((i & 127u) == 127u) {
            uint32_t t;
            asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
            t = __shfl_sync(0xffffffffu, t, 0);
            if (i == 127u)
                t0 = t;
            else if (t - t0 > (uint32_t)kWaitNs)
                return false;
        }
    }
    return false;
}

__device__ __forceinline__ constexpr float power2(int e) { return e < 0 ? 1.f / (1 << -e) : (float)(1 << e); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// v[r] joined over the lanes by op, for all R rows at once: lane i ends with
// row i % R in v[0].  Each step halves the rows of a lane, R - 1 exchanges;
// then lanes of the same row meet.
template <int R, typename Op>
__device__ __forceinline__ void lane_reduce(float (&v)[R], int lane, Op op)
{
#pragma unroll
    for (int h = R / 2; h; h >>= 1) {
        const bool up = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + h], h);
            v[i] = op(up ? v[i + h] : v[i], got);
        }
    }
#pragma unroll
    for (int h = R; h < 32; h <<= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], h));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// a - b of two pairs of fp16.
__device__ __forceinline__ uint32_t half2_less(uint32_t a, uint32_t b)
{
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// Two floats as E4M3 codes (a in the low byte), and back.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3_values(uint32_t c)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y)
{
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Columns (rows of a group) c0 .. c0 + n - 1 at `col` of S^T, the terms of
// their queries joined: n = 8, or 16 with fewer waits.
template <bool FP8, int RW, int n>
__device__ __forceinline__ void load_logits(uint32_t col, float (&x)[n])
{
    if constexpr (!FP8) {
        if constexpr (n == 8)
            tmem_ld8(col, x);
        else
            tmem_ld16(col, x);
    } else if constexpr (RW < 8) {  // both terms lie in 8 columns
        tmem_ld8(col, x);
#pragma unroll
        for (int i = 0; i < RW; ++i) x[i] = fmaf(x[RW + i], 0.0625f, x[i]);
    } else {
        float y[n];
        tmem_ld_pair(col, col + RW, x, y);
#pragma unroll
        for (int i = 0; i < n; ++i) x[i] = fmaf(y[i], 0.0625f, x[i]);
    }
}

// ceil(log2) of a page's V scale, from the append's smallest on: a scale of 0 (a
// page that is not there is read as zeros, its scales too) must not draw the
// reference so far down that the weights overflow.
__device__ __forceinline__ float scale_log2(float sv)
{
    const uint32_t u = __float_as_uint(sv) & 0x7fffffffu;
    return (float)max((int)(u >> 23) - 127 + ((u & 0x7fffffu) != 0), kEMin);
}

// 8 columns of O^T at `col`, the terms of their weights joined.  An infinity in
// V is one in the first term's sum alone: the second, 0 or less, makes it NaN.
template <bool FP8, int RW>
__device__ __forceinline__ void load_out(uint32_t col, float (&x)[8])
{
    auto join = [](float a, float b) { return FP8 || fabsf(a) <= 3.402823466e38f ? a + b : a; };
    if constexpr (RW < 8) {  // all terms lie in 8 columns
        tmem_ld8(col, x);
#pragma unroll
        for (int i = 0; i < RW; ++i) x[i] = join(x[i], FP8 ? x[RW + i] + x[2 * RW + i] : x[RW + i]);
    } else {
        float y[8];
        tmem_ld_pair(col, col + RW, x, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = join(x[i], y[i]);
        if constexpr (FP8) {
            tmem_ld8(col + 2 * RW, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] += y[i];
        }
    }
}

// Two fp16 weights, rounded to 9 bits, as three E5M2 numbers each, in the upper
// bytes of the fp16 halves: 3 bits from the top of what is left, the
// differences exact.  What is below 2^-16 is cut off.
__device__ __forceinline__ void cut_weights(__half2 w, uint32_t (&t)[3])
{
    const uint32_t u = (*reinterpret_cast<const uint32_t *>(&w) + 0x00020002u) & 0xfffcfffcu;
    t[0] = u & 0xff00ff00u;
    const uint32_t rest = half2_less(u, t[0]);
    t[1] = rest & 0xff00ff00u;
    t[2] = half2_less(rest, t[1]);
}

// Half a step of what the cut leaves, 2^-16: numbers below 2^-6 are rounded by
// it instead of cut off, so that thousands of them do not lose the same part.
// Above, it moves a number by 2^-11 of it at the most.
constexpr float kHalfCut = 0x1p-17f;

// The producer warp of a kernel of shape S.  Returns the copies it issued.
template <typename S, bool FP8, int RB>
__device__ __forceinline__ int produce(const CUtensorMap *map, const AttnParams &p, long long x0, long long x1, int seq,
                                       long long base, uint32_t sbase, uint32_t full, uint32_t empty)
{
    const int lane = threadIdx.x & 31;
    int issued = 0;
    // Producer: the parts of the tiles, a copy per page, in the order in
    // which the MMA warp takes them (K of a tile before V of the one
    // before it), and the pages' scales with K.
    Walk<RB> walk(p, x0, x1, seq, base);
    Item it;
    const int ppt = kTile >> p.b.page_log2;  // pages of a tile
    const uint32_t page_bytes = (uint32_t)S::C * 128 << p.b.page_log2;
    const int groups_log2 = p.b.page_log2 - 3;  // 8-key groups of a page
    const int none = (p.b.num_pages * p.Hk) << groups_log2;  // first group past the tensor: reads as zeros
    bool ok = true;
    // Part `part` of the `pages` pages that lane i < pages names by its first group.
    auto load = [&](int part, int group0, int pages, const float *scale, int g) {
        const int st = issued % S::SLOTS;
        const uint32_t bar = full + 8 * st;
        if (issued >= S::SLOTS) {
            ok = wait_poll(empty + 8 * st, (uint32_t)(issued / S::SLOTS - 1) & 1u, p.wait_limit);
            if (!ok) return;
        }
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)pages * page_bytes);
        __syncwarp();
        const uint32_t dst = sbase + st * S::SLOT;
        if (lane < pages) tma_load_4d(dst + lane * page_bytes, map, 0, 0, part * S::C, group0, bar);
        if (FP8) {
            if (lane < pages)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(
                                 sbase + S::OFF_SC + (g % kScaleRing) * 64 + lane * 8),
                             "l"(scale), "r"(group0 < none ? 8 : 0)
                             : "memory");
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        }
        ++issued;
    };
    int g = 0, before = 0, pages_before = 0;
    while (ok && walk.next(it)) {
        const int32_t *table = p.b.table + (size_t)it.seq * p.b.width;
        const int last = (block_limit<RB>(walk.q, p, it.rb) - 1) >> p.b.page_log2;  // last page
        int page = lane < ppt && it.t0 * ppt + lane <= last ? __ldg(table + it.t0 * ppt + lane) : 0;
        for (int t = it.t0; t < it.t1; ++t) {
            const int pages = min(ppt, last + 1 - t * ppt);
            const int mine = page, ahead = (t + 1) * ppt + lane;
            if (lane < ppt && t + 1 < it.t1 && ahead <= last) page = __ldg(table + ahead);
            const bool held = mine >= 0 && mine < p.b.num_pages;
            if (!held && lane < pages) atomicOr(p.b.status, ST_CHECK);
            const int group0 = held ? (mine * p.Hk + it.head) << groups_log2 : none;
            load(0, group0, pages, FP8 ? p.scales + ((size_t)(held ? mine : 0) * p.Hk + it.head) * 2 : nullptr, g);
            if (S::PARTS == 2) {
                if (ok && g > 0) load(1, before, pages_before, nullptr, 0);
                before = group0;
                pages_before = pages;
            }
            if (!ok) break;
            ++g;
        }
    }
    if (S::PARTS == 2 && ok && g > 0) load(1, before, pages_before, nullptr, 0);
    if (!ok && lane == 0) atomicOr(p.b.status, ST_TIMEOUT);
    if (FP8) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    return issued;
}

// What the other warps are told of an item (have: or that there is none).
template <int RB>
__device__ __forceinline__ void put_info(Info &f, const Item &cur, int nr, bool have, bool more, const AttnParams &p, int workers, long long total)
{
    f.nr = nr;
    f.t0 = have ? cur.t0 : 0;
    f.t1 = have ? cur.t1 : 0;
    f.more = more;
    if (have) {
        const Seq q = {cur.row, cur.n, cur.len, false};
        f.limit = block_limit<RB>(q, p, cur.rb);
        f.least = cur.len - cur.n + p.over_g(cur.rb * RB) + 1;
        f.first = blockIdx.x;
        f.pieces = 1;
        if (cur.split()) {
            // The CTA whose run [total c / workers, ..) holds place x: the last with total c / workers <= x.
            f.first = (int)(((cur.x + 1) * workers + total - 1) / total) - 1;
            f.pieces = (int)(((cur.x + (long long)(cur.tiles - 1) * cur.weight + 1) * workers + total - 1) / total) - f.first;
        }
    }
}

// Adds a piece of a shared item to its counter; the last of them leaves it at
// 0 for the next launch.
__device__ __forceinline__ bool arrive(int *counter, int pieces)
{
    const bool last = atomicAdd(counter, 1) == pieces - 1;
    if (last) *counter = 0;
    return last;
}

// Joins the pieces of row r of an item whose first piece is of CTA cf, in the
// order of their keys; one warp.  The pieces' (m, l) lie across its lanes, 32
// pieces at a time, and its lanes read `ahead` pieces of O ahead.
template <int D, int RB, int ahead>
__device__ __forceinline__ void join_row(const float *work, int piece, int cf, int pieces, int r, __nv_bfloat16 *out)
{
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    float top = kNoMax, sum = 0.f, o[V] = {};
    for (int i0 = 0; i0 < pieces; i0 += 32) {
        const int n = min(32, pieces - i0), i = i0 + lane;
        const float *src = work + (size_t)(2 * (cf + i) + (i > 0)) * piece + RB * D + r;
        const float mi = lane < n ? __ldcg(src) : kNoMax, li = lane < n ? __ldcg(src + RB) : 0.f;
        const float now = fmaxf(top, warp_max(mi)), f = ex2(top - now), w = ex2(mi - now);
        top = now;
        sum = fmaf(sum, f, warp_sum(lane < n ? w * li : 0.f));
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] *= f;
#pragma unroll(ahead)
        for (int j = 0; j < n; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const float *at = work + (size_t)(2 * (cf + i0 + j) + (i0 + j > 0)) * piece + r * D + lane * V;
            if constexpr (V == 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(at));
                o[0] = fmaf(wj, x.x, o[0]);
                o[1] = fmaf(wj, x.y, o[1]);
                o[2] = fmaf(wj, x.z, o[2]);
                o[3] = fmaf(wj, x.w, o[3]);
            } else {
                const float2 x = __ldcg(reinterpret_cast<const float2 *>(at));
                o[0] = fmaf(wj, x.x, o[0]);
                o[1] = fmaf(wj, x.y, o[1]);
            }
        }
    }
    __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>(out + lane * V);
    const float inv = 1.f / sum;
#pragma unroll
    for (int v = 0; v < V; v += 2) dst[v / 2] = __floats2bfloat162_rn(o[v] * inv, o[v + 1] * inv);
}

// 8 elements of a query row as two numbers each, E4M3 and then E4M3 of 16 times
// the rest, or (`plain`) E5M2 of the rest: 3 bits hold it, 8 bits less 4 rounded,
// exactly where the first has its 4.  x = (t1 + t2 / 16 or t1 + t2) times the
// returned scale 2^e, the smallest with every element of the row at most
// 448 2^e; below 2^-6 of it the rest loses no more than 2^-14, 2^-21 of the row's
// largest.  The row's other elements are in the TR - 1 lanes beside.  A row with
// an infinity or NaN has the scale NaN.
template <int TR, bool plain>
__device__ __forceinline__ float split_query(const uint4 &x, uint32_t (&a)[4], uint32_t (&b)[4])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8], top = 0.f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
        finite = finite && fabsf(v[j]) <= 3.402823466e38f;
        top = fmaxf(top, fabsf(v[j]));
    }
    if (!finite) top = INFINITY;
#pragma unroll
    for (int o = 1; o < TR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t u = __float_as_uint(top);
    const int e = max((int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u), -110);
    const float inv = top < INFINITY ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float y0 = v[2 * j] * inv, y1 = v[2 * j + 1] * inv;
        a[j] = e4m3_pair(y0, y1);
        const float2 t = e4m3_values(a[j]);
        if (plain)
            b[j] = __nv_cvt_float2_to_fp8x2(make_float2(y0 - t.x, y1 - t.y), __NV_SATFINITE, __NV_E5M2);
        else
            b[j] = e4m3_pair((y0 - t.x) * 16.f, (y1 - t.y) * 16.f);
    }
    return top < INFINITY ? __uint_as_float((uint32_t)(127 + e) << 23) : NAN;
}

// This CTA's run of the cost line, and the sequence (with its first place)
// that holds its beginning.  `total` is divided over `workers` CTAs, so few
// that a tile begins in every run inside an item.  All threads call
// it; sequences that do not fit are reported.
template <int RB, int kThreads>
__device__ void find_run(const AttnParams &p, long long &x0, long long &x1, int &seq, long long &base, long long &total,
                         int &workers)
{
    __shared__ long long wsum[kThreads / 32];
    __shared__ long long f_base;
    __shared__ int f_seq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long incl = 0, mine = 0;
    // Inclusive prefix of the costs of sequences s0 + tid; returns their sum.
    auto scan = [&](int s0) {
        const int s = s0 + tid;
        mine = 0;
        if (s < p.b.n_seqs) {
            const Seq q = load_seq(p.b, s);
            if (q.bad && blockIdx.x == 0) atomicOr(p.b.status, ST_CHECK);
            mine = seq_cost<RB>(q, p);
        }
        incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        __syncthreads();
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        long long sum = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) incl += wsum[w];
            sum += wsum[w];
        }
        return sum;
    };
    total = 0;
    for (int s0 = 0; s0 < p.b.n_seqs; s0 += kThreads) total += scan(s0);
    const long long most = (total + kLeastRun<RB> - 1) / kLeastRun<RB>;
    workers = most < gridDim.x ? (int)most : (int)gridDim.x;
    x0 = x1 = 0;
    if ((int)blockIdx.x < workers) {
        x0 = total * blockIdx.x / workers;
        x1 = total * (blockIdx.x + 1) / workers;
    }
    if (x0 < x1) {
        long long before = 0;
        for (int s0 = 0;; s0 += kThreads) {
            const long long sum = p.b.n_seqs <= kThreads ? total : scan(s0);
            const long long first = before + incl - mine;
            if (x0 >= first && x0 < first + mine) {
                f_seq = s0 + tid;
                f_base = first;
            }
            before += sum;
            if (x0 < before) break;
        }
        __syncthreads();
        seq = f_seq;
        base = f_base;
    }
}

// A CTA whose waits gave up adds its pieces all the same: a counter left
// part-way would make a later launch join pieces that are not there yet.  All
// threads call it, after the CTA's last barrier; it finds the run anew, which
// then need not be kept in registers for it.
template <int RB, int kThreads, int groups>
__device__ __noinline__ void arrive_late(const AttnParams &p, const int *arrived)
{
    long long x0, x1, base = 0, total;
    int seq = 0, workers;
    find_run<RB, kThreads>(p, x0, x1, seq, base, total, workers);
    if (threadIdx.x != 0) return;
    Walk<RB> walk(p, x0, x1, seq, base);
    Item it;
    Info f;
    for (int j = 0; walk.next(it);) {
        if (!it.split()) continue;
        put_info<RB>(f, it, 0, true, false, p, workers, total);
        for (int i = 0; i < groups; ++i)
            if (j >= arrived[i]) arrive(p.counters + f.first * groups + i, f.pieces);
        ++j;
    }
}

template <bool FP8, int D, int RB>
__global__ void __launch_bounds__(Shape<FP8, D, RB>::THREADS, Shape<FP8, D, RB>::CTAS)
    attn_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ AttnParams p)
{
    using S = Shape<FP8, D, RB>;
    constexpr int NS = S::NS, NO = S::NO, SLOTS = S::SLOTS;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char *const smem = smem_raw + (sbase - raw);
    const uint32_t full = sbase + S::OFF_BAR, empty = full + 8 * SLOTS;
    const uint32_t q_ready = empty + 8 * SLOTS, i_free = q_ready + 8 * S::QD;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp >= S::SOFT ? min((warp - S::SOFT) / 4, S::GROUPS - 1) : warp >= 1 && warp <= S::GROUPS ? warp - 1 : 0;
    // of the warp's group
    const uint32_t s_full = i_free + 8 * S::QD + group * 56, p_ready = s_full + 16, pv_done = s_full + 32, drain = s_full + 48;
    float *const rows = reinterpret_cast<float *>(smem + S::OFF_ROW);
    constexpr int RS = RB < 8 ? 8 : RB;                              // stride of the rows' arrays
    float *const qc = rows;                                          // [QD][RS] logit factor of a row
    int *const bound = reinterpret_cast<int *>(rows + S::QD * RS);   // [QD][RS] keys a row attends
    uint32_t *const orow = reinterpret_cast<uint32_t *>(rows + 2 * S::QD * RS);  // [QD][RS] its (token, head)
    // Of each group, rows counted from the group's first (the groups may be at different items):
    constexpr int GS = S::RW < 8 ? 8 : S::RW;
    float *const wmax = rows + 3 * S::QD * RS + group * 18 * GS;     // [2][4][GS] largest of a softmax warp, by tile parity
    float *const lsum = wmax + 8 * GS;                               // [2][4][GS] sums of weights, by item parity
    float *const mref = lsum + 8 * GS;                               // [2][GS] references, by item parity
    Info *const info = reinterpret_cast<Info *>(smem + S::OFF_INFO);
    Shared &sh = *reinterpret_cast<Shared *>(info + S::QD);

    if (threadIdx.x == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(full + 8 * s, FP8 ? 33 : 1);  // expect_tx, and for E4M3 the page scales' copies of each lane
            mbar_init(empty + 8 * s, S::GROUPS);
        }
        for (int i = 0; i < S::GROUPS; ++i) {
            const uint32_t g0 = s_full + i * 56;
            for (int j = 0; j < 2; ++j) {
                mbar_init(g0 + 8 * j, 1);           // s_full
                mbar_init(g0 + 16 + 8 * j, 4);      // p_ready: one arrival a warp
                mbar_init(g0 + 32 + 8 * j, 1);      // pv_done
            }
            mbar_init(g0 + 48, 1);                  // drain
        }
        for (int i = 0; i < S::QD; ++i) {
            mbar_init(q_ready + 8 * i, 1);
            mbar_init(i_free + 8 * i, 4 * S::GROUPS);
        }
        sh.arrived[0] = sh.arrived[1] = sh.gave_up = 0;
        fence_barrier_init();
        prefetch_tmap(&map);
    }
    if (warp == 2) {
        tmem_alloc(smem_u32(&sh.tmem), S::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    pdl_wait();
    pdl_launch_dependents();
    long long x0, x1, base = 0, total;
    int seq = 0, workers;
    find_run<RB, S::THREADS>(p, x0, x1, seq, base, total, workers);
    int issued = 0;

    if (warp == 0) {
        issued = produce<S, FP8, RB>(&map, p, x0, x1, seq, base, sbase, full, empty);
    } else if (warp <= S::GROUPS) {
        // MMA warp of a group: all lanes keep the (uniform) books, one elected lane
        // issues; a lone lane in a branch would make the compiler move every
        // operand to the uniform registers inside it, MMA by MMA.
        constexpr uint32_t id_s = FP8 ? idesc_e4m3_f32(128, NS) : idesc_bf16_f32(128, NS);
        constexpr uint32_t id_o = (FP8 ? idesc_e4m3_f32(128, NO) | kIdescBE5M2 : idesc_bf16_f32(128, NO)) | kIdescAMMajor;
        const bool leader = elect_one();
        const uint32_t s_col = tmem + group * S::GCOLS, o_col = s_col + 2 * NS;
        int g = 0, taken = 0, slot_before = 0;
        bool ok = true, first_before = false;
        uint32_t o_before = 0;
        auto mma = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
            if (FP8)
                umma_e4m3(d, a, b, idesc, acc);
            else
                umma_bf16(d, a, b, idesc, acc);
        };
        auto wait = [&](uint32_t bar, uint32_t parity) { return wait_poll(bar, parity, p.wait_limit); };
        // O^T (+)= V^T w of tile `g`.
        auto values = [&](int g) {
            const uint32_t b = g & 1;
            int st = slot_before;
            if (S::PARTS == 2) {
                st = taken % SLOTS;
                if (!wait(full + 8 * st, (uint32_t)(taken / SLOTS) & 1u)) return false;
                ++taken;
            }
            if (!wait(p_ready + 8 * b, (uint32_t)(g >> 1) & 1u)) return false;
            tc_fence_after();
            const uint64_t pd = sw128_kmajor_desc(sbase + S::OFF_P + b * S::PBUF + group * S::PGROUP);
            const uint64_t vd = sw128_mmajor_desc(sbase + st * S::SLOT + S::VCOL, 1024, S::SBO);
            if (leader) {
#pragma unroll
                for (int s = 0; s < kTile * S::EB / 32; ++s)
                    mma(o_before, vd + (uint64_t)(s * (32 / S::EB / 8) * S::SBO / 16),
                        pd + (uint64_t)((s / 4 * S::PROWS * 128 + s % 4 * 32) / 16), id_o, !(first_before && s == 0));
                umma_commit(empty + 8 * st);
                umma_commit(pv_done + 8 * b);
            }
            __syncwarp();
            return true;
        };
        for (int k = 0; ok; ++k) {
            const int buf = k % S::QD;
            ok = wait(q_ready + 8 * buf, (uint32_t)(k / S::QD) & 1u);
            if (!ok) break;
            const int t0 = __shfl_sync(0xffffffffu, info[buf].t0, 0), t1 = __shfl_sync(0xffffffffu, info[buf].t1, 0);
            if (t1 == 0) break;
            for (int t = t0; t < t1; ++t) {
                const int st = taken % SLOTS;
                ok = wait(full + 8 * st, (uint32_t)(taken / SLOTS) & 1u);
                if (!ok) break;
                ++taken;
                tc_fence_after();
                const uint64_t kd = sw128_kmajor_desc(sbase + st * S::SLOT, S::SBO);
                const uint64_t qd = sw128_kmajor_desc(sbase + S::OFF_Q + buf * S::QBUF + group * S::QGROUP);
                if (leader) {
#pragma unroll
                    for (int s = 0; s < D * S::EB / 32; ++s)
                        mma(s_col + (g & 1) * NS, kd + (uint64_t)((s / 4 * 1024 + s % 4 * 32) / 16),
                            qd + (uint64_t)((s / 4 * S::QROWS * 128 + s % 4 * 32) / 16), id_s, s > 0);
                    if (S::PARTS == 2) umma_commit(empty + 8 * st);
                    umma_commit(s_full + 8 * (g & 1));
                }
                __syncwarp();
                if (g > 0 && !(ok = values(g - 1))) break;
                slot_before = st;
                first_before = t == t0;
                o_before = o_col + (k & 1) * NO;
                ++g;
            }
        }
        if (ok && g > 0) ok = values(g - 1);
        if (!ok && leader) atomicOr(p.b.status, ST_TIMEOUT);
        if (leader) {
            umma_commit(drain);  // every MMA issued has completed before the tensor memory is freed
            drain_phase(drain, 0);
        }
        __syncwarp();
    } else if (warp == S::QUERY) {
        // Query warp: writes each item's rows as the B operand of S^T, their
        // constants and the item's Info, ahead of the softmax warps.
        const float kScale = rsqrtf((float)D) * 1.4426950408889634f;
        constexpr int TR = D / 8;       // lanes of a row, 8 elements each
        constexpr int kPass = 32 / TR;  // rows at once
        const int c = lane % TR;
        Walk<RB> walk(p, x0, x1, seq, base);
        Item it, next;
        bool more = walk.next(it), ok = true;
        for (int k = 0;; ++k) {
            const int buf = k % S::QD;
            const uint32_t q0 = sbase + S::OFF_Q + buf * S::QBUF;
            const Item cur = it;
            const bool have = more;
            const int nr = have ? min(RB, cur.n * p.G - cur.rb * RB) : 0;
            const int half = S::GROUPS == 1 ? RB : (nr + 15) / 16 * 8;  // rows of the first group
            auto fetch = [&](int r) {
                const int rr = cur.rb * RB + r, i = p.over_g(rr);
                return r < nr ? *reinterpret_cast<const uint4 *>(
                                    p.q + ((size_t)(cur.row + i) * p.Hq + cur.head * p.G + rr - i * p.G) * D + c * 8)
                              : make_uint4(0, 0, 0, 0);
            };
            constexpr int AT = RB / kPass < 1 ? 1 : RB / kPass > 4 ? 4 : RB / kPass;  // passes in hand
            uint4 x[AT];
#pragma unroll
            for (int i = 0; i < AT; ++i) x[i] = fetch(i * kPass + lane / TR);
            if (have) more = walk.next(next);
            if (k >= S::QD) {
                ok = wait_poll(i_free + 8 * buf, (uint32_t)(k / S::QD - 1) & 1u, p.wait_limit);
                if (!ok) break;
            }
            for (int r0 = 0; r0 < nr; r0 += AT * kPass) {
#pragma unroll
                for (int i = 0; i < AT; ++i) {
                    const int r = r0 + i * kPass + lane / TR;
                    if (r0 + i * kPass >= nr) break;
                    if (FP8) {
                        uint32_t a[4], b[4];
                        const float scale = split_query<TR, false>(x[i], a, b);
                        if (r < nr) {
                            const int r1 = r < half ? r : r - half, r2 = S::RW + r1;
                            const uint32_t to = q0 + (r < half ? 0 : S::QGROUP) + (c & 1) * 8;
                            sts64(to + r1 * 128 + (((c >> 1) ^ (r1 & 7)) << 4), a[0] | a[1] << 16, a[2] | a[3] << 16);
                            sts64(to + r2 * 128 + (((c >> 1) ^ (r2 & 7)) << 4), b[0] | b[1] << 16, b[2] | b[3] << 16);
                            if (c == 0) qc[buf * RS + r] = kScale * scale;
                        }
                    } else if (r < nr) {
                        const int r1 = r < half ? r : r - half;
                        sts128(q0 + (r < half ? 0 : S::QGROUP) + (c >> 3) * S::QROWS * 128 + r1 * 128 + (((c & 7) ^ (r1 & 7)) << 4), x[i]);
                        if (c == 0) qc[buf * RS + r] = kScale;
                    }
                }
                if (r0 + AT * kPass < nr) {
#pragma unroll
                    for (int i = 0; i < AT; ++i) x[i] = fetch(r0 + (AT + i) * kPass + lane / TR);
                }
            }
            for (int r = lane; r < RB; r += 32) {
                const int rr = cur.rb * RB + r, i = p.over_g(rr);
                bound[buf * RS + r] = r < nr ? cur.len - cur.n + i + 1 : 0;
                orow[buf * RS + r] = (uint32_t)(cur.row + i) * (uint32_t)p.Hq + (uint32_t)(cur.head * p.G + rr - i * p.G);
                if (r >= nr) qc[buf * RS + r] = 0.f;  // of a last pair or chunk, beyond the block
            }
            if (lane == 0) put_info<RB>(info[buf], cur, nr, have, have && more, p, workers, total);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready + 8 * buf);
            if (!have) break;
            it = next;
        }
        if (!ok && lane == 0) atomicOr(p.b.status, ST_TIMEOUT);
        __syncwarp();
    } else {
        // Softmax warps: thread = key of a tile (TMEM lane of S^T) with RW
        // rows of the block in registers, and element of head_dim in the
        // epilogue (lane of O^T).
        constexpr int RW = S::RW;
        constexpr int GR = RW < 8 ? RW : RW == 8 ? 4 : 8;  // rows that are taken or left together
        const int wg = (warp - S::SOFT) % 4;  // warp of the group
        const int tid = threadIdx.x - 32 * S::SOFT - group * kSoft;
        // First row of the group: each takes half of a block's rows, in eights.
        auto first_row = [&](int nr) { return group == 0 ? 0 : (nr + 15) / 16 * 8; };
        auto group_rows = [&](int nr) { return S::GROUPS == 1 ? nr : group == 0 ? min(nr, (nr + 15) / 16 * 8) : nr - first_row(nr); };
        const uint32_t bar = kSoftBar + group;
        const int L = (warp & 3) * 32 + lane;
        const int e = L - (128 - D);  // element of the row; head_dim 64: lanes 64 .. 127
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16) + group * S::GCOLS;
        const float kScale = rsqrtf((float)D) * 1.4426950408889634f;
        bool fail = false;
        int g = 0;

        // Writes the rows of item k, whose last tile is number gl, or its
        // piece of them; runs behind the first tile of the next item.
        auto epilogue = [&](int k, int gl) {
            const Info &f = info[k % S::QD];
            const int nr = group_rows(f.nr), R0 = first_row(f.nr), pieces = f.pieces, cf = f.first;
            const float *ls = lsum + (k & 1) * 4 * GS;
            const float *ms = mref + (k & 1) * GS;
            const uint32_t *to = orow + k % S::QD * RS + R0;
            fail = fail || !wait_poll(pv_done + 8 * (gl & 1), (uint32_t)(gl >> 1) & 1u, p.wait_limit);
            tc_fence_after();
            float *const piece = p.work + (size_t)(2 * blockIdx.x + ((int)blockIdx.x > cf)) * S::PIECE;
            // Lane r: the sum of row r.
            const float sum = lane < nr ? ls[lane] + ls[GS + lane] + ls[2 * GS + lane] + ls[3 * GS + lane] : 1.f;
            const float scale = (pieces == 1 ? 1.f / sum : 1.f) * power2(-S::HELD);
#pragma unroll
            for (int c0 = 0; c0 < RW; c0 += 8) {
                if (c0 >= nr) break;
                float o[8];
                load_out<FP8, RW>(trow + 2 * NS + (k & 1) * NO + c0, o);
#pragma unroll
                for (int i = 0; i < 8 && i < RW; ++i) {
                    const int r = c0 + i;
                    o[i] *= __shfl_sync(0xffffffffu, scale, r);
                    if (r < nr && e >= 0) {
                        if (pieces == 1)
                            p.out[(size_t)to[r] * D + e] = __float2bfloat16_rn(o[i]);
                        else
                            __stcg(piece + (R0 + r) * D + e, o[i]);
                    }
                }
            }
            if (pieces > 1 && wg == 0 && lane < nr) {
                __stcg(piece + RB * D + R0 + lane, ms[lane]);
                __stcg(piece + RB * (D + 1) + R0 + lane, sum);
            }
            tc_fence_before();
            if (pieces > 1) {
                // Each group publishes and joins its own rows.
                __threadfence();
                named_bar_sync(bar, kSoft);
                if (tid == 0) {
                    sh.last[group] = arrive(p.counters + cf * S::GROUPS + group, pieces);
                    ++sh.arrived[group];
                }
                named_bar_sync(bar, kSoft);
                if (sh.last[group]) {
                    // Joins the pieces in the order of their keys.
                    __threadfence();
                    for (int r = wg; r < nr; r += 4)
                        join_row<D, RB, RW <= 8 ? 8 : 4>(p.work, S::PIECE, cf, pieces, R0 + r, p.out + (size_t)to[r] * D);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(i_free + 8 * (k % S::QD));
        };

        for (int k = 0;; ++k) {
            const int buf = k % S::QD;
            fail = fail || !wait_poll(q_ready + 8 * buf, (uint32_t)(k / S::QD) & 1u, p.wait_limit);
            if (named_bar_or(bar, kSoft, fail)) break;
            const int t0 = info[buf].t0, t1 = info[buf].t1, nr = group_rows(info[buf].nr), R0 = first_row(info[buf].nr);
            if (t1 == 0) {
                if (k > 0) epilogue(k - 1, g - 1);
                break;
            }
            const int limit = info[buf].limit, least = info[buf].least, more = info[buf].more;
            const float *qcb = qc + buf * RS + R0;
            const int *bnd = bound + buf * RS + R0;
            const uint32_t o_col = trow + 2 * NS + (k & 1) * NO;
            // Sums of weights, and references.
            float *const ms = mref + (k & 1) * GS;
            float l[RW], mr[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) l[r] = mr[r] = 0.f;
            uint32_t open = (1u << nr) - 1;  // rows whose reference no logit has set yet: any above -infinity will
            bool stop = false;
            for (int t = t0; t < t1; ++t, ++g) {
                const int b = g & 1;
                const int key = t * kTile + L;
                float *const wm = wmax + b * 4 * GS;
                fail = fail || !wait_poll(s_full + 8 * b, (uint32_t)(g >> 1) & 1u, p.wait_limit);
                float sk = 1.f, sv = 1.f, ev = 0.f;
                if (FP8 && key < limit) {
                    // S^T is there, so K's barrier had completed, and the copies of its page scales with it.
                    const float2 sc = *reinterpret_cast<const float2 *>(smem + S::OFF_SC + g % kScaleRing * 64 +
                                                                        (L >> p.b.page_log2) * 8);
                    sk = sc.x;
                    sv = sc.y;
                    ev = scale_log2(sv);
                }
                tc_fence_after();
                const bool whole = (t + 1) * kTile <= least;  // no row of the block is masked
                // y: logits (log2) less the row's reference so far (0 at the first tile); masked ones are -inf.
                float y[RW];
                constexpr int CH = RW < 16 ? 8 : 16;
#pragma unroll
                for (int c0 = 0; c0 < RW; c0 += CH) {
                    if (c0 >= nr) break;
                    float x[CH];
                    load_logits<FP8, RW>(trow + b * NS + c0, x);
#pragma unroll
                    for (int i = 0; i < CH && i < RW; ++i) {
                        if (i % GR == 0 && c0 + i >= nr) break;
                        const int r = c0 + i;
                        if constexpr (RW < 4) {
                            y[r] = fmaf(x[i], FP8 ? qcb[r] * sk : kScale, -mr[r]);
                        } else if (i % 4 == 0) {
                            float4 c4 = make_float4(kScale, kScale, kScale, kScale);
                            const float4 m4 = make_float4(mr[r], mr[r + 1], mr[r + 2], mr[r + 3]);
                            if (FP8) c4 = *reinterpret_cast<const float4 *>(qcb + r);
                            y[r] = fmaf(x[i], FP8 ? c4.x * sk : kScale, -m4.x);
                            y[r + 1] = fmaf(x[i + 1], FP8 ? c4.y * sk : kScale, -m4.y);
                            y[r + 2] = fmaf(x[i + 2], FP8 ? c4.z * sk : kScale, -m4.z);
                            y[r + 3] = fmaf(x[i + 3], FP8 ? c4.w * sk : kScale, -m4.w);
                        }
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        if (r % GR == 0 && r >= nr) break;
                        if (key >= bnd[r]) y[r] = -INFINITY;
                    }
                }
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int r = 0; r < RW; ++r) {
                    if (r % GR == 0 && r >= nr) break;
                    tops[r % 4] = fmaxf(tops[r % 4], y[r]);
                }
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                bool need = t == t0 || open;
                if (!need) need = named_bar_or(bar, kSoft, top > (float)(S::SLACK + S::LOW) - ev || fail);
                if (need) {
                    // New references: each row's largest logit + log2(V scale), where that has grown past the slack.
                    float v[RW];
#pragma unroll
                    for (int r = 0; r < RW; ++r) v[r] = y[r] + (mr[r] + ev);
                    lane_reduce(v, lane, [](float a, float c) { return fmaxf(a, c); });
                    if (lane < nr) wm[wg * GS + lane] = v[0];
                    if (named_bar_or(bar, kSoft, fail)) {
                        stop = true;
                        break;
                    }
                    if (t > t0) fail = fail || !wait_poll(pv_done + 8 * (b ^ 1), (uint32_t)((g - 1) >> 1) & 1u, p.wait_limit);
                    tc_fence_after();
                    uint32_t shut = 0;
#pragma unroll
                    for (int c0 = 0; c0 < RW; c0 += 8) {
                        if (c0 >= nr) break;
                        constexpr int W = RW < 8 ? RW : 8;
                        float f[8], best[W];
                        bool any = false;
#pragma unroll
                        for (int i = 0; i < W; i += W < 4 ? W : 4) {
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const float *src = wm + w * GS + c0 + i;
                                if constexpr (W < 4) {
#pragma unroll
                                    for (int j = 0; j < W; ++j) best[j] = w == 0 ? src[j] : fmaxf(best[j], src[j]);
                                } else {
                                    const float4 x = *reinterpret_cast<const float4 *>(src);
                                    best[i] = w == 0 ? x.x : fmaxf(best[i], x.x);
                                    best[i + 1] = w == 0 ? x.y : fmaxf(best[i + 1], x.y);
                                    best[i + 2] = w == 0 ? x.z : fmaxf(best[i + 2], x.z);
                                    best[i + 3] = w == 0 ? x.w : fmaxf(best[i + 3], x.w);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            const int r = c0 + i;
                            f[i] = 1.f;
                            if (i % GR == 0 && r >= nr) break;
                            // rows beyond the block never ask for more (and weigh nothing)
                            const float held = mr[r], old = open >> r & 1 ? -INFINITY : held, low = best[i] - (float)S::LOW;
                            const bool grow = low > old + (float)S::SLACK && r < nr;
                            const float now = r >= nr ? kNever : grow ? low : held;
                            if (grow) f[i] = ex2(old - now), any = true;
                            shut |= (uint32_t)grow << r;
                            y[r] += held - now;
                            mr[r] = now;
                            l[r] *= f[i];
                        }
                        if (any && t > t0) {
                            float o[8];
                            if constexpr (RW >= 8) {
                                float o2[8];
                                tmem_ld_pair(o_col + c0, o_col + RW + c0, o, o2);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[i] *= f[i], o2[i] *= f[i];
                                tmem_st8(o_col + c0, o);
                                tmem_st8(o_col + RW + c0, o2);
                                if constexpr (FP8) {
                                    tmem_ld8(o_col + 2 * RW + c0, o);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) o[i] *= f[i];
                                    tmem_st8(o_col + 2 * RW + c0, o);
                                }
                            } else {  // with fewer than 8 rows all terms are in these columns
                                tmem_ld8(o_col + c0, o);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[i] *= f[i % W];
                                tmem_st8(o_col + c0, o);
                            }
                        }
                    }
                    open &= ~shut;
                }
                // The buffer of the weights is free once tile g - 2 is done.
                if (g >= 2) fail = fail || !wait_poll(pv_done + 8 * b, (uint32_t)((g - 2) >> 1) & 1u, p.wait_limit);
                // Row n of the weights' operand, this key's element: 128 n bytes on, with the 16-byte column of a row turned by
                // its number in 8 (the swizzle).
                const uint32_t key_at = S::OFF_P + b * S::PBUF + group * S::PGROUP +
                                        (FP8 ? (uint32_t)L : (uint32_t)(L >> 6) * S::PROWS * 128 + (L & 63) * 2);
                auto at = [&](int n) { return smem + (key_at ^ ((n & 7) << 4)) + n * 128; };
                const float hold = sv * power2(S::HELD);
#pragma unroll
                for (int r = 0; r < RW; r += 2) {
                    if (r % GR == 0 && r >= nr) break;
                    const float w0 = ex2(y[r]), w1 = ex2(y[r + 1]);
                    l[r] += w0;
                    l[r + 1] += w1;
                    if (FP8) {
                        uint32_t terms[3];
                        cut_weights(__floats2half2_rn(fmaf(w0, hold, kHalfCut), fmaf(w1, hold, kHalfCut)), terms);
#pragma unroll
                        for (int i = 0; i < 3; ++i) {
                            *at(i * RW + r) = (unsigned char)(terms[i] >> 8);
                            *at(i * RW + r + 1) = (unsigned char)(terms[i] >> 24);
                        }
                    } else {
                        // w = t1 + t2, to 2^-16 of it
                        const __nv_bfloat162 h = __floats2bfloat162_rn(w0, w1);
                        const __nv_bfloat162 c = __floats2bfloat162_rn(w0 - __low2float(h), w1 - __high2float(h));
                        *reinterpret_cast<__nv_bfloat16 *>(at(r)) = h.x;
                        *reinterpret_cast<__nv_bfloat16 *>(at(r + 1)) = h.y;
                        *reinterpret_cast<__nv_bfloat16 *>(at(RW + r)) = c.x;
                        *reinterpret_cast<__nv_bfloat16 *>(at(RW + r + 1)) = c.y;
                    }
                }
                if ((t + 1) * kTile > limit) {
                    // Behind the last key that a row attends: whatever the slot holds, its weight of 0 meets zeros (both
                    // groups write them, each before its own product).
                    const int pos = S::PARTS == 1 ? g : t + 1 < t1 || more ? 2 * g + 2 : 2 * g + 1;
                    fail = fail || !wait_poll(full + 8 * (pos % SLOTS), (uint32_t)(pos / SLOTS) & 1u, p.wait_limit);
                    if (key >= limit) {
                        const uint32_t row = sbase + pos % SLOTS * S::SLOT + (L >> 3) * S::SBO + (L & 7) * 128;
                        const uint4 z = make_uint4(0, 0, 0, 0);
                        if (FP8 && D == 64) {
#pragma unroll
                            for (int c = 4; c < 8; ++c) sts128(row + ((c ^ (L & 7)) << 4), z);
                        } else {
#pragma unroll
                            for (int i = S::PARTS == 1 ? 1 : 0; i < S::C; ++i)
#pragma unroll
                                for (int c = 0; c < 8; ++c) sts128(row + i * 1024 + c * 16, z);
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + 8 * b);
                if (t == t0 && k > 0) epilogue(k - 1, g - 1);
            }
            if (stop) break;
            lane_reduce(l, lane, [](float a, float c) { return a + c; });
            if (lane < nr) lsum[((k & 1) * 4 + wg) * GS + lane] = l[0];
            if (tid == 0) {
#pragma unroll
                for (int r = 0; r < RW; ++r)
                    if (r < nr) ms[r] = open >> r & 1 ? kNoMax : mr[r];
            }
        }
        if (fail) {
            atomicOr(p.b.status, ST_TIMEOUT);
            sh.gave_up = 1;
        }
    }

    __syncthreads();
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < SLOTS && s < issued; ++s)  // every copy issued has landed
            drain_phase(full + 8 * s, (uint32_t)((issued - 1 - s) / SLOTS) & 1u);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, S::TMEM);
    }
    if (sh.gave_up) arrive_late<RB, S::THREADS, S::GROUPS>(p, sh.arrived);
}

// ---------------------------------------------------------------------------
// Many rows of a sequence and KV head: blocks of 128, rows as the wide operand.
//
//     S  = Q K^T    [128 rows x 128 keys]      (tcgen05.mma, M = rows)
//     O += w V      [128 rows x head_dim]      (M = rows, w from tensor memory)
//
// A thread owns half of a row of S (two threads a row, 64 keys each): its
// maximum and sum need no other lane, and the weights go back to tensor memory
// over the logits they came from.  The two halves of the keys have references,
// sums and accumulators of their own, which meet at the item's end: nothing is
// agreed upon in between, and one half's warps wait while the other's count.
//
// A tile keeps the tensor cores busy for 4 * 128 * 128 * head_dim operations
// (540 to 1080 clocks); its softmax, read from tensor memory, counted and
// written back, takes a warp about 2000.  That chain is the bound (16% of the
// tensor pipe's cycles busy at heads of 64, 36% in E4M3; without the
// exponentials it would take 5% less): two warps a scheduler are all that the
// registers of 64 keys a thread allow.  One sequence x 4096 tokens over 16384
// keys, 32 heads over 8 of 128, bf16: 660 us, 1458 TFLOP/s; 32 sequences of
// 4000 to 8196 keys x 20 to 64 rows, E4M3: 140.9 us, 0.43 of the copy bandwidth.
// The two halves taking whole tiles in turn, each thread a row of 128 keys,
// took 193 us there when this form took 134.
//
// bf16: a weight is rounded to one bf16 number, 2^-8 of it, as the values beside
// it and the result are.  A second term costs what the tensor cores have no room
// for: 2 x 4096 tokens, 32 heads over 8 of 128, 277 us with one and 358 with
// two; 4096 tokens over 20480 keys 854 and 1161; 2 x 2048 tokens, 24 heads over 8
// of 64, 72 and 78.
//
// E4M3: the queries' two terms are accumulated into the same S, the second
// unscaled and so E5M2, for its range.  A weight is cut as above,
// without a conversion instruction (conversions to E4M3 and back took as long as
// the exponentials) or a scale between the terms: one accumulator.  Off by at
// most 2^-9 of the weight plus 2^-26 of the reference; a NaN becomes a zero
// there, and the row is NaN by its sum.
template <bool FP8, int D>
struct Rows {
    static constexpr int RB = 128;
    static constexpr int EB = FP8 ? 1 : 2;
    static constexpr int TERMS = FP8 ? 2 : 1;    // of a query row
    static constexpr int WTERMS = FP8 ? 3 : 1;   // of a weight
    static constexpr int THREADS = 384;      // producer, MMA, 2 query, 8 softmax warps
    static constexpr int CTAS = 1;
    static constexpr int QD = 2;
    static constexpr int PARTS = D * EB == 256 ? 2 : 1;
    static constexpr int C = 2 * D * EB / 128 / PARTS;
    static constexpr uint32_t SLOT = C * kBox;
    static constexpr uint32_t SBO = C * 1024;
    // V in its part: a column of its own, or (E4M3, 64) the second half of K's,
    // which then gives O columns that nobody reads before its own.
    static constexpr uint32_t VCOL = PARTS == 2 || (FP8 && D == 64) ? 0 : 1024;
    static constexpr int NO = FP8 || D == 128 ? 128 : 64;   // columns of a half's accumulator
    static constexpr int O0 = FP8 && D == 64 ? 64 : 0;      // first of V's
    static constexpr int QBOXES = D * EB < 128 ? 1 : D * EB / 128;
    static constexpr uint32_t QTERM = QBOXES * kBox, QBUF = TERMS * QTERM;
    static constexpr int TMEM = 512;                         // S twice, O of the two halves
    static constexpr int SLACK = FP8 ? 6 : 8, LOW = FP8 ? kLow : 0, HELD = FP8 ? 15 - SLACK - LOW : 0;  // fp16 reaches 2^16
    static constexpr int PIECE = RB * (D + 2);
    static constexpr uint32_t ROWF = (3 * QD + 4 + 4) * RB;  // qc, bound, orow [QD], refs [2][2], sums [2][2]
    static constexpr uint32_t FIXED = QD * QBUF + kBarBytes + kScaleRing * 64 + ROWF * 4 + QD * sizeof(Info) + sizeof(Shared) + 1024;
    static constexpr uint32_t ROOM = 228 * 1024 - 1024 - 256;
    static constexpr int SLOTS = (ROOM - FIXED) / SLOT > 8 ? 8 : (ROOM - FIXED) / SLOT;
    static constexpr uint32_t OFF_Q = SLOTS * SLOT;
    static constexpr uint32_t OFF_BAR = OFF_Q + QD * QBUF;
    static constexpr uint32_t OFF_SC = OFF_BAR + kBarBytes;
    static constexpr uint32_t OFF_ROW = OFF_SC + kScaleRing * 64;
    static constexpr uint32_t OFF_INFO = OFF_ROW + ROWF * 4;
    static constexpr uint32_t SMEM = OFF_INFO + QD * sizeof(Info) + sizeof(Shared) + 1024;
    static_assert(SLOTS >= PARTS + 1 && (2 * SLOTS + 11 + 2 * QD) * 8 <= (int)kBarBytes, "slots of K and V");
    static_assert(SMEM <= ROOM, "shared memory of a CTA");
};

template <bool FP8, int D>
__global__ void __launch_bounds__(Rows<FP8, D>::THREADS, 1)
    rows_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ AttnParams p)
{
    using S = Rows<FP8, D>;
    constexpr int SLOTS = S::SLOTS, RB = S::RB, NO = S::NO;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char *const smem = smem_raw + (sbase - raw);
    const uint32_t full = sbase + S::OFF_BAR, empty = full + 8 * SLOTS;
    const uint32_t q_ready = empty + 8 * SLOTS, i_free = q_ready + 8 * S::QD;
    const uint32_t s_full = i_free + 8 * S::QD, p_ready = s_full + 16, pv_done = s_full + 48;  // [half][parity]
    const uint32_t drain = s_full + 80;
    float *const qc = reinterpret_cast<float *>(smem + S::OFF_ROW);            // [QD][RB] logit factor of a row
    int *const bound = reinterpret_cast<int *>(qc + S::QD * RB);               // [QD][RB] keys a row attends
    uint32_t *const orow = reinterpret_cast<uint32_t *>(qc + 2 * S::QD * RB);  // [QD][RB] its (token, head)
    float *const refs = qc + 3 * S::QD * RB;                                   // [2][2][RB] by item parity and half
    float *const sums = refs + 4 * RB;                                         // [2][2][RB] by item parity and half
    Info *const info = reinterpret_cast<Info *>(smem + S::OFF_INFO);
    Shared &sh = *reinterpret_cast<Shared *>(info + S::QD);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(full + 8 * s, FP8 ? 33 : 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(p_ready + 8 * i, 4);  // one arrival a softmax warp
            mbar_init(pv_done + 8 * i, 1);
        }
        mbar_init(drain, 1);
        for (int i = 0; i < S::QD; ++i) {
            mbar_init(q_ready + 8 * i, 2);  // one arrival a query warp
            mbar_init(i_free + 8 * i, 8);
        }
        sh.arrived[0] = sh.arrived[1] = sh.gave_up = 0;
        fence_barrier_init();
        prefetch_tmap(&map);
    }
    if (warp == 3) {
        tmem_alloc(smem_u32(&sh.tmem), S::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t o_col = tmem + 256;

    pdl_wait();
    pdl_launch_dependents();
    long long x0, x1, base = 0, total;
    int seq = 0, workers;
    find_run<RB, S::THREADS>(p, x0, x1, seq, base, total, workers);
    int issued = 0;

    if (warp == 0) {
        issued = produce<S, FP8, RB>(&map, p, x0, x1, seq, base, sbase, full, empty);
    } else if (warp == 1) {
        constexpr uint32_t id_s = FP8 ? idesc_e4m3_f32(128, 128) : idesc_bf16_f32(128, 128);
        constexpr uint32_t id_o = (FP8 ? idesc_e4m3_f32(128, NO) | kIdescAE5M2 : idesc_bf16_f32(128, NO)) | kIdescBNMajor;
        const bool leader = elect_one();
        int g = 0, taken = 0, slot_before = 0;
        bool ok = true, first_before = false;
        auto wait = [&](uint32_t bar, uint32_t parity) { return wait_poll(bar, parity, p.wait_limit); };
        // O (+)= w V of tile `g`.
        auto values = [&](int g) {
            const uint32_t b = g & 1;
            int st = slot_before;
            if (S::PARTS == 2) {
                st = taken % SLOTS;
                if (!wait(full + 8 * st, (uint32_t)(taken / SLOTS) & 1u)) return false;
                ++taken;
            }
            const uint64_t vd = sw128_mmajor_desc(sbase + st * S::SLOT + S::VCOL, 1024, S::SBO);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!wait(p_ready + 16 * half + 8 * b, (uint32_t)(g >> 1) & 1u)) return false;
                tc_fence_after();
                if (leader) {
                    constexpr int kSteps = kTile / 2 * S::EB / 32;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const uint64_t v = vd + (uint64_t)((half * kSteps + s) * (32 / S::EB / 8) * S::SBO / 16);
                        const uint32_t at = tmem + b * 128 + half * 64 + s * 8, o = o_col + half * 128;
                        const uint32_t acc = !(first_before && s == 0);
                        if (FP8) {
#pragma unroll
                            for (int term = 0; term < S::WTERMS; ++term) umma_e4m3_ta(o, at + 16 * term, v, id_o, acc || term > 0);
                        } else {
                            umma_bf16_ta(o, at, v, id_o, acc);
                        }
                    }
                    if (half == 1) umma_commit(empty + 8 * st);
                    umma_commit(pv_done + 16 * half + 8 * b);
                }
                __syncwarp();
            }
            return true;
        };
        for (int k = 0; ok; ++k) {
            const int buf = k % S::QD;
            ok = wait(q_ready + 8 * buf, (uint32_t)(k / S::QD) & 1u);
            if (!ok) break;
            const int t0 = __shfl_sync(0xffffffffu, info[buf].t0, 0), t1 = __shfl_sync(0xffffffffu, info[buf].t1, 0);
            if (t1 == 0) break;
            for (int t = t0; t < t1; ++t) {
                const int st = taken % SLOTS;
                ok = wait(full + 8 * st, (uint32_t)(taken / SLOTS) & 1u);
                if (!ok) break;
                ++taken;
                tc_fence_after();
                const uint64_t kd = sw128_kmajor_desc(sbase + st * S::SLOT, S::SBO);
                const uint64_t qd = sw128_kmajor_desc(sbase + S::OFF_Q + buf * S::QBUF);
                if (leader) {
                    constexpr int kSteps = D * S::EB / 32;
#pragma unroll
                    for (int s = 0; s < kSteps * S::TERMS; ++s) {
                        const int i = s % kSteps;
                        const uint64_t q = qd + (uint64_t)((s / kSteps * S::QTERM + i / 4 * kBox + i % 4 * 32) / 16);
                        const uint64_t key = kd + (uint64_t)((i / 4 * 1024 + i % 4 * 32) / 16);
                        if (FP8)
                            umma_e4m3(tmem + (g & 1) * 128, q, key, s < kSteps ? id_s : id_s | kIdescAE5M2, s > 0);
                        else
                            umma_bf16(tmem + (g & 1) * 128, q, key, id_s, s > 0);
                    }
                    if (S::PARTS == 2) umma_commit(empty + 8 * st);
                    umma_commit(s_full + 8 * (g & 1));
                }
                __syncwarp();
                if (g > 0 && !(ok = values(g - 1))) break;
                slot_before = st;
                first_before = t == t0;
                ++g;
            }
        }
        if (ok && g > 0) ok = values(g - 1);
        if (!ok && leader) atomicOr(p.b.status, ST_TIMEOUT);
        if (leader) {
            umma_commit(drain);
            drain_phase(drain, 0);
        }
        __syncwarp();
    } else if (warp <= 3) {
        // Query warps: rows of a block as the A operand of S, by asynchronous copies (bf16, passes in turn) or through
        // registers that split them (E4M3, every other AT passes each, the first before the buffer is free; 16 of them
        // spilled, and long sequences took 4% more).
        const float kScale = rsqrtf((float)D) * 1.4426950408889634f;
        constexpr int TR = D / 8, kPass = 32 / TR, AT = FP8 ? 8 : 1;
        const int c = lane % TR, first = (warp - 2) * AT * kPass;
        Walk<RB> walk(p, x0, x1, seq, base);
        Item it, next;
        bool more = walk.next(it), ok = true;
        for (int k = 0;; ++k) {
            const int buf = k % S::QD;
            const uint32_t q0 = sbase + S::OFF_Q + buf * S::QBUF;
            const Item cur = it;
            const bool have = more;
            const int nr = have ? min(RB, cur.n * p.G - cur.rb * RB) : 0;
            auto source = [&](int r) {
                const int rr = cur.rb * RB + r, i = p.over_g(rr);
                return p.q + ((size_t)(cur.row + i) * p.Hq + cur.head * p.G + rr - i * p.G) * D + c * 8;
            };
            auto fetch = [&](int r) { return r < nr ? *reinterpret_cast<const uint4 *>(source(r)) : make_uint4(0, 0, 0, 0); };
            uint4 x[AT];
            if (FP8) {
#pragma unroll
                for (int i = 0; i < AT; ++i) x[i] = fetch(first + i * kPass + lane / TR);
            }
            if (have) more = walk.next(next);
            if (k >= S::QD) {
                ok = wait_poll(i_free + 8 * buf, (uint32_t)(k / S::QD - 1) & 1u, p.wait_limit);
                if (!ok) break;
            }
            if (!FP8) {
                for (int r = (warp - 2) * kPass + lane / TR; r < nr; r += 2 * kPass)
                    cp_async16(q0 + (c >> 3) * kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4), source(r));
            }
            for (int r0 = first; FP8 && r0 < nr; r0 += 2 * AT * kPass) {
#pragma unroll
                for (int i = 0; i < AT; ++i) {
                    const int r = r0 + i * kPass + lane / TR;
                    if (r0 + i * kPass >= nr) break;
                    uint32_t a[4], b[4];
                    const float scale = split_query<TR, true>(x[i], a, b);
                    const uint32_t to = q0 + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8;
                    sts64(to, a[0] | a[1] << 16, a[2] | a[3] << 16);
                    sts64(to + S::QTERM, b[0] | b[1] << 16, b[2] | b[3] << 16);
                    if (c == 0) qc[buf * RB + r] = kScale * scale;
                }
                if (r0 + 2 * AT * kPass < nr) {
#pragma unroll
                    for (int i = 0; i < AT; ++i) x[i] = fetch(r0 + (2 * AT + i) * kPass + lane / TR);
                }
            }
            for (int r = lane + 32 * (warp - 2); r < RB; r += 64) {
                const int rr = cur.rb * RB + r, i = p.over_g(rr);
                bound[buf * RB + r] = r < nr ? cur.len - cur.n + i + 1 : 0;
                if (!FP8) qc[buf * RB + r] = kScale;
                orow[buf * RB + r] = (uint32_t)(cur.row + i) * (uint32_t)p.Hq + (uint32_t)(cur.head * p.G + rr - i * p.G);
            }
            if (warp == 2 && lane == 0) put_info<RB>(info[buf], cur, nr, have, have && more, p, workers, total);
            if (!FP8) asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready + 8 * buf);
            if (!have) break;
            it = next;
        }
        if (!ok && lane == 0) atomicOr(p.b.status, ST_TIMEOUT);
        __syncwarp();
    } else if (warp >= 4) {
        const int half = (warp - 4) / 4, sw = warp - 4;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        // A wait that gave up is dealt with where all meet, at the items' ends; until then the warp goes on without
        // waiting.
        bool fail = false;
        int g = 0;
        for (int k = 0;; ++k) {
            const int buf = k % S::QD;
            fail = fail || !wait_poll(q_ready + 8 * buf, (uint32_t)(k / S::QD) & 1u, p.wait_limit);
            if (named_bar_or(kSoftBar, 256, fail)) break;
            const int t0 = info[buf].t0, t1 = info[buf].t1, nr = info[buf].nr, limit = info[buf].limit, least = info[buf].least;
            const int more = info[buf].more, pieces = info[buf].pieces, cf = info[buf].first;
            if (t1 == 0) break;
            const float c = row < nr ? qc[buf * RB + row] : 0.f;
            const int bnd = bound[buf * RB + row];
            float m = 0.f, l = 0.f;
            bool open = row < nr;  // no logit has set the reference yet: any above -infinity will
            for (int t = t0; t < t1; ++t, ++g) {
                const int b = g & 1;
                const int key0 = t * kTile + half * 64;
                fail = fail || !wait_poll(s_full + 8 * b, (uint32_t)(g >> 1) & 1u, p.wait_limit);
                tc_fence_after();
                const uint32_t s_col = trow + b * 128 + half * 64;
                // Page scales of the half's four runs of 16 keys.
                float sk[4], sv[4], ev[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sk[j] = sv[j] = 1.f;
                    ev[j] = 0.f;
                    if (FP8 && key0 + 16 * j < limit) {
                        const float2 sc = *reinterpret_cast<const float2 *>(smem + S::OFF_SC + g % kScaleRing * 64 +
                                                                            ((half * 64 + 16 * j) >> p.b.page_log2) * 8);
                        sk[j] = sc.x;
                        sv[j] = sc.y;
                        ev[j] = scale_log2(sc.y);
                    }
                }
                // y: logits (log2) less the reference so far; masked ones are -inf.
                float y[64], top = -INFINITY;
                tmem_ld64(s_col, y);
#pragma unroll
                for (int j = 0; j < 64; j += 2) fma_pair(y[j], y[j + 1], FP8 ? c * sk[j / 16] : c, -m);
                if ((t + 1) * kTile > least) {
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (key0 + j >= bnd) y[j] = -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float a = y[16 * j], d = y[16 * j + 1];
#pragma unroll
                    for (int i = 2; i < 16; i += 2) {
                        a = fmaxf(a, y[16 * j + i]);
                        d = fmaxf(d, y[16 * j + i + 1]);
                    }
                    top = fmaxf(top, fmaxf(a, d) + ev[j]);
                }
                const bool grow = top > (open ? -INFINITY : (float)(S::SLACK + S::LOW));
                if (__any_sync(0xffffffffu, grow)) {
                    // A new reference where the largest logit + log2(V scale) of the row has grown past the slack.
                    const float d = grow ? top - (float)S::LOW : 0.f;
                    m += d;
#pragma unroll
                    for (int j = 0; j < 64; ++j) y[j] -= d;
                    if (t > t0) {
                        const float f = open && grow ? 0.f : ex2(-d);
                        l *= f;
                        fail = fail || !wait_poll(pv_done + 16 * half + 8 * (b ^ 1), (uint32_t)((g - 1) >> 1) & 1u, p.wait_limit);
                        __syncwarp();
                        tc_fence_after();
                        const uint32_t at = trow + 256 + S::O0 + half * 128;
                        for (int i = 0; i < D; i += 16) {
                            float o[16];
                            tmem_ld16(at + i, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] *= f;
                            tmem_st16(at + i, o);
                        }
                    }
                    if (grow) open = false;
                }
                // Weights, over the logits they come from.
                if (FP8) {
                    float terms[3][16];
#pragma unroll
                    for (int j = 0; j < 64; j += 4) {
                        const float hold = sv[j / 16] * power2(S::HELD);
                        uint32_t a[3], d[3];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float w0 = ex2(y[j + 2 * i]), w1 = ex2(y[j + 2 * i + 1]);
                            l += w0 + w1;
                            cut_weights(__floats2half2_rn(fmaf(w0, hold, kHalfCut), fmaf(w1, hold, kHalfCut)), i == 0 ? a : d);
                        }
#pragma unroll
                        for (int term = 0; term < 3; ++term) terms[term][j / 4] = __uint_as_float(__byte_perm(a[term], d[term], 0x7531));
                    }
#pragma unroll
                    for (int term = 0; term < 3; ++term) tmem_st16(s_col + 16 * term, terms[term]);
                } else {
                    float held[32];
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        const float w0 = ex2(y[j]), w1 = ex2(y[j + 1]);
                        l += w0 + w1;
                        const __nv_bfloat162 h = __floats2bfloat162_rn(w0, w1);
                        held[j / 2] = __uint_as_float(*reinterpret_cast<const uint32_t *>(&h));
                    }
                    tmem_st32(s_col, held);
                }
                if ((t + 1) * kTile > limit) {
                    // Behind the last key that a row attends: whatever the slot holds, its weight of 0 meets zeros.
                    const int pos = S::PARTS == 1 ? g : t + 1 < t1 || more ? 2 * g + 2 : 2 * g + 1;
                    fail = fail || !wait_poll(full + 8 * (pos % SLOTS), (uint32_t)(pos / SLOTS) & 1u, p.wait_limit);
                    if ((row >> 6) == half && t * kTile + row >= limit) {
                        const uint32_t at = sbase + pos % SLOTS * S::SLOT + (row >> 3) * S::SBO + (row & 7) * 128;
                        const uint4 z = make_uint4(0, 0, 0, 0);
                        if (FP8 && D == 64) {
#pragma unroll
                            for (int i = 4; i < 8; ++i) sts128(at + ((i ^ (row & 7)) << 4), z);
                        } else {
#pragma unroll
                            for (int x = S::PARTS == 1 ? 1 : 0; x < S::C; ++x)
#pragma unroll
                                for (int i = 0; i < 8; ++i) sts128(at + x * 1024 + i * 16, z);
                        }
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + 16 * half + 8 * b);
            }

            // ---- the item's rows, or its piece of them; half of the columns each
            refs[((k & 1) * 2 + half) * RB + row] = open ? kNoMax : m;
            sums[((k & 1) * 2 + half) * RB + row] = l;
            for (int i = 0; i < 2; ++i)
                fail = fail || !wait_poll(pv_done + 16 * i + 8 * ((g - 1) & 1), (uint32_t)((g - 1) >> 1) & 1u, p.wait_limit);
            if (named_bar_or(kSoftBar, 256, fail)) break;
            tc_fence_after();
            const float *const ms = refs + (k & 1) * 2 * RB + row, *const ls = sums + (k & 1) * 2 * RB + row;
            const float ref = fmaxf(ms[0], ms[RB]);
            float f0 = ex2(ms[0] - ref), f1 = ex2(ms[RB] - ref);
            const float sum = fmaf(ls[RB], f1, ls[0] * f0);
            const float scale = (pieces == 1 ? 1.f / sum : 1.f) * power2(-S::HELD);
            f0 *= scale;
            f1 *= scale;
            float *const piece = p.work + (size_t)(2 * blockIdx.x + ((int)blockIdx.x > cf)) * S::PIECE;
            const uint32_t *const to = orow + buf * RB;
            __nv_bfloat16 *const dst = p.out + (size_t)to[row] * D + half * (D / 2);
#pragma unroll
            for (int i = 0; i < D / 2; i += 16) {
                float o[16];
                const uint32_t at = trow + 256 + S::O0 + half * (D / 2) + i;
                float o1[16];
                tmem_ld_pair(at, at + 128, o, o1);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = fmaf(o1[j], f1, o[j] * f0);
                if (row < nr) {
#pragma unroll
                    for (int j = 0; j < 16; j += 8) {
                        if (pieces == 1) {
                            uint32_t w[4];
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(o[j + 2 * v], o[j + 2 * v + 1]);
                                w[v] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            *reinterpret_cast<uint4 *>(dst + i + j) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
                            float4 *const at4 = reinterpret_cast<float4 *>(piece + row * D + half * (D / 2) + i + j);
                            __stcg(at4, make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]));
                            __stcg(at4 + 1, make_float4(o[j + 4], o[j + 5], o[j + 6], o[j + 7]));
                        }
                    }
                }
            }
            tc_fence_before();
            if (pieces > 1) {
                if (half == 0) {
                    __stcg(piece + RB * D + row, ref);
                    __stcg(piece + RB * (D + 1) + row, sum);
                }
                __threadfence();
                named_bar_sync(kSoftBar, 256);
                if (sw == 0 && lane == 0) {
                    sh.last[0] = arrive(p.counters + cf, pieces);
                    ++sh.arrived[0];
                }
                named_bar_sync(kSoftBar, 256);
                if (sh.last[0]) {
                    __threadfence();
                    for (int r = sw; r < nr; r += 8)
                        join_row<D, RB, 4>(p.work, S::PIECE, cf, pieces, r, p.out + (size_t)to[r] * D);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(i_free + 8 * buf);
        }
        if (fail) {
            atomicOr(p.b.status, ST_TIMEOUT);
            sh.gave_up = 1;
        }
    }

    __syncthreads();
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < SLOTS && s < issued; ++s)  // every copy issued has landed
            drain_phase(full + 8 * s, (uint32_t)((issued - 1 - s) / SLOTS) & 1u);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, S::TMEM);
    }
    if (sh.gave_up) arrive_late<RB, S::THREADS, 1>(p, sh.arrived);
}

}  // namespace dsa_paged_k

using dsa_detail::cuda_fail;
using dsa_detail::dev_alloc;
using dsa_detail::fail;

namespace {

using namespace dsa_paged_k;

// One instantiation of the kernel on the handle's device: calls
// fn(kernel, shared memory, floats of a published piece, CTAs per SM, threads).
template <bool FP8, int D, int RB, typename Fn>
int with_shape(Fn &&fn)
{
    using S = Shape<FP8, D, RB>;
    return fn(attn_kernel<FP8, D, RB>, (int)S::SMEM, S::PIECE, S::CTAS, S::THREADS);
}

template <typename Fn>
int with_kernel(const dsa_paged_ctx *h, int rb, Fn &&fn)
{
    const bool eight = h->dtype == DSA_FP8_E4M3;
    auto rows = [&](auto eight_c, auto d_c) {
        constexpr bool E = decltype(eight_c)::value;
        constexpr int D = decltype(d_c)::value;
        switch (rb) {
        case 2: return with_shape<E, D, 2>(fn);
        case 8: return with_shape<E, D, 8>(fn);
        case 16: return with_shape<E, D, 16>(fn);
        default: break;
        }
        if constexpr (E)
            if (rb == 32) return with_shape<E, D, 32>(fn);
        using S = Rows<E, D>;
        return fn(rows_kernel<E, D>, (int)S::SMEM, S::PIECE, S::CTAS, S::THREADS);
    };
    using std::integral_constant;
    if (h->D == 128)
        return eight ? rows(std::true_type(), integral_constant<int, 128>()) : rows(std::false_type(), integral_constant<int, 128>());
    return eight ? rows(std::true_type(), integral_constant<int, 64>()) : rows(std::false_type(), integral_constant<int, 64>());
}

// Row blocks: the smallest that holds max_new new tokens of a group's heads is
// launched (128 for more).  A block of 32 is built for E4M3 only.  Its tiles
// cost their rows, those of 128 rows the same for any number.  Heads of 128,
// 32 over 8, block of 32 against 128: 32 sequences x 8000 keys x 20 rows 129 and
// 162 us, 32 x 4000 x 32 rows 89 and 97, 32 x 600 x 24 rows 34 and 29, 96 x 300 x
// 32 rows 67 and 53; heads of 64, 32 x 4000 x 24 rows 74 and 90.  In bf16 128 was
// faster everywhere, with weights of one term in both: 165 and 164 us, 96 and 94,
// 34.5 and 25.5, 62 and 45, 63 and 58.  For 33 to 64 rows a block of 64 took longer
// than 128 (4 x 2000 keys x 64 rows: 54 us against 31 in E4M3, 45 against 27 in
// bf16).
constexpr int kBlocks[5] = {2, 8, 16, 32, 128};

int block_index(const dsa_paged_ctx *h, long long rows)
{
    int i = 0;
    while (i < 4 && rows > kBlocks[i]) ++i;
    return i == 3 && h->dtype != DSA_FP8_E4M3 ? 4 : i;
}

}  // namespace

int dsa_detail::paged_attn_init(dsa_paged_ctx *h)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    cudaDriverEntryPointQueryResult found;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", (void **)&encode, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess || found != cudaDriverEntryPointSuccess || !encode)
        return fail(DSA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const bool eight = h->dtype == DSA_FP8_E4M3;
    // Columns of 128 bytes: (byte in the column, key of 8, column, group of 8
    // keys), so that a box of a page's keys lands with 8 keys of each column
    // in turn, whatever the page size.
    const cuuint64_t row = 2ull * h->D * (eight ? 1 : 2);  // bytes of a token's K and V
    const cuuint64_t dims[4] = {eight ? 128u : 64u, 8, row / 128, (cuuint64_t)h->num_pages * h->Hk * (h->page / 8)};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {eight ? 128u : 64u, 8, row == 512 ? 2 : (cuuint32_t)(row / 128), (cuuint32_t)(h->page / 8)};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = encode(&h->map, eight ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, h->pages, dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(DSA_ERR_CUDA, "cuTensorMapEncodeTiled (pages) failed (%d)", (int)r);

    size_t work = 0;
    for (int i = 0; i < 5; ++i) {
        int rc = with_kernel(h, kBlocks[i], [&](auto kernel, int smem, int piece, int ctas, int) {
            cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (err != cudaSuccess) return cuda_fail(err, "paged attention kernel attribute (is this an sm_103 device?)");
            // The occupancy query of the runtime answers 1 for these kernels; launch bounds, shared and tensor memory
            // are laid out for `ctas`, and nothing waits on another CTA.
            h->grid[i] = ctas * h->sms < kMaxGrid ? ctas * h->sms : kMaxGrid;
            const size_t need = (size_t)2 * h->grid[i] * piece;
            work = need > work ? need : work;
            return (int)DSA_OK;
        });
        if (rc != DSA_OK) return rc;
    }
    int rc = dev_alloc((void **)&h->work, work * sizeof(float), "paged attention pieces");
    if (rc == DSA_OK) rc = dev_alloc((void **)&h->counters, kCounters * sizeof(int), "paged attention counters");
    if (rc == DSA_OK && (e = cudaMemset(h->counters, 0, kCounters * sizeof(int))) != cudaSuccess) rc = cuda_fail(e, "cudaMemset");
    return rc;
}

int dsa_detail::paged_attn_launch(dsa_paged_ctx *h, const dsa_paged_k::Batch &b, int max_new, const void *q, void *out,
                                  cudaStream_t st)
{
    AttnParams p;
    p.b = b;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.scales = h->scales;
    p.work = h->work;
    p.counters = h->counters;
    p.Hq = h->Hq;
    p.Hk = h->Hk;
    p.G = h->Hq / h->Hk;
    p.g_mul = p.G > 1 && ((long long)b.n_tokens + 128) * p.G * p.G < (1LL << 32) ? (uint32_t)(((1ULL << 32) + p.G - 1) / p.G) : 0;
    p.wait_limit = h->wait_limit;
    p.lead = h->D / 16;
    const long long rows = (long long)(max_new < b.n_tokens ? max_new : b.n_tokens) * p.G;
    const int i = block_index(h, rows);
    return with_kernel(h, kBlocks[i], [&](auto kernel, int smem, int, int, int threads) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(h->grid[i]);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, h->map, p);
        return err == cudaSuccess ? (int)DSA_OK : cuda_fail(err, "paged attention launch");
    });
}
