// attend.cuh -- what the kernels of tree attention share: how the work is cut, how tiles of the paged cache
// come into shared memory, where results go.
//
// The cut.  All tiles of all sequences and heads of keys lie in a row, which is cut into equal parts, one for
// each CTA that the GPU holds at once (a team of CTAs, where the rows of a head of keys need several).  A part that
// begins or ends inside a sequence leaves its sums in scratch memory, and a second kernel joins them in their
// order.  So one long sequence fills the GPU, and ragged ones leave no SM idle.  Each sequence and head counts
// BEGIN tiles more than it has, for its queries, its nodes and its output: without them short sequences that lie
// side by side became one CTA's (16 trees of which one has no context: 257 us, 126 without that one).
#pragma once

#include <cuda.h>

#include "ops_internal.cuh"

namespace gbper {
namespace attend {

typedef unsigned long long u64;
constexpr int kRecord = 8;             // ints of a CTA's record for the joining kernel
// barriers by the numbers of AttendArgs::withhold: one that waits for an arrival more than come, to test what follows
enum Barrier { kKeys = 1, kValues, kRelease, kMeet, kQueries, kScores, kP, kOutputs };

// ---- how the work is cut -----------------------------------------------------------------------
struct Span {              // a sequence
    int len, total, count; // context, context and nodes, nodes; in the table's range
    bool bad;
};

__device__ __forceinline__ Span span(const AttendArgs &a, unsigned b)
{
    const long long room = (long long)a.c.width * a.c.page.d;
    const int len = a.lens[b], count = a.counts ? a.counts[b] : (int)a.nodes;
    Span s;
    s.bad = len < 0 || count < 0 || (unsigned)count > a.nodes || (long long)len + count > room;
    s.count = min(max(count, 0), (int)a.nodes);
    s.len = (int)min((long long)max(len, 0), room);
    s.total = (int)min((long long)s.len + s.count, room);
    return s;
}

template <int KT>
__device__ __forceinline__ unsigned tiles_of(const Span &s)
{
    return s.count == 0 ? 1u : max(1u, ((unsigned)s.total + KT - 1) / KT);   // a sequence without nodes has zeros to write
}

// x / y by 32 bits where they are enough (a division of 64 bits takes some hundred cycles)
__device__ __forceinline__ u64 divide(u64 x, u64 y)
{
    return (x | y) >> 32 ? x / y : (u64)((unsigned)x / (unsigned)y);
}

// A team's stretches, one sequence and head after another.
template <int KT, unsigned BEGIN>
struct Walk {
    u64 pos, end, at;        // in tiles, BEGIN before each sequence's and head's; at: where the sequence begins
    u64 size, more;          // tiles of a team; the first `more` teams have one more
    unsigned b, n_tiles, h, tile0, tile1;
    Span s;

    // All NT threads of the CTA; `scan` holds NT / 32 words.  False: the team has nothing to do.
    template <int NT>
    __device__ __forceinline__ bool begin(const AttendArgs &a, unsigned team, unsigned max_teams, u64 *scan)
    {
        const unsigned t = threadIdx.x, lane = t & 31u, warp = t >> 5;
        const unsigned per = (a.batch + NT - 1) / NT;
        const unsigned b0 = min(t * per, a.batch), b1 = min(b0 + per, a.batch);
        u64 mine = 0;
        for (unsigned i = b0; i < b1; ++i) mine += tiles_of<KT>(span(a, i)) + BEGIN;
        u64 upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const u64 o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        u64 before = upto - mine, all = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            if (w < (int)warp) before += scan[w];
            all += scan[w];
        }
        all *= a.c.heads;
        before *= a.c.heads;                                   // tiles in front of this thread's sequences
        size = divide(all, max_teams);
        more = all - size * max_teams;
        pos = team * size + min((u64)team, more);
        end = pos + size + (team < more);
        if (pos >= end) return false;
        __syncthreads();
        if (pos >= before && pos < before + mine * a.c.heads) {   // one thread's
            unsigned i = b0;
            u64 x = before;
            for (;; ++i) {
                const u64 n = (u64)(tiles_of<KT>(span(a, i)) + BEGIN) * a.c.heads;
                if (pos < x + n) break;
                x += n;
            }
            scan[0] = i;
            scan[1] = x;
        }
        __syncthreads();
        b = (unsigned)scan[0];
        at = scan[1];
        s = span(a, b);
        n_tiles = tiles_of<KT>(s);
        return true;
    }

    // One sequence and head for the whole cluster, its tiles shared among `parts` CTAs.
    __device__ __forceinline__ void one(const AttendArgs &a, unsigned seq, unsigned head, unsigned rank, unsigned parts)
    {
        b = seq;
        h = head;
        s = span(a, b);
        n_tiles = tiles_of<KT>(s);
        tile0 = (unsigned)((u64)rank * n_tiles / parts);
        tile1 = (unsigned)((u64)(rank + 1) * n_tiles / parts);
    }

    __device__ __forceinline__ bool next(const AttendArgs &a)
    {
        do {
            if (pos >= end) return false;
            if (pos >= at + (u64)(n_tiles + BEGIN) * a.c.heads) {
                at += (u64)(n_tiles + BEGIN) * a.c.heads;
                ++b;
                s = span(a, b);
                n_tiles = tiles_of<KT>(s);
            }
            const unsigned whole = n_tiles + BEGIN;
            h = (unsigned)divide(pos - at, whole);
            const unsigned x0 = (unsigned)(pos - at - (u64)h * whole), x1 = (unsigned)min((u64)whole, x0 + (end - pos));
            tile0 = x0 > BEGIN ? x0 - BEGIN : 0;
            tile1 = x1 > BEGIN ? x1 - BEGIN : 0;
            pos += x1 - x0;
        } while (tile0 == tile1);
        return true;
    }

    __device__ __forceinline__ bool part() const { return tile0 != 0 || tile1 < n_tiles; }

    // the record of a CTA that begins what others end
    __device__ __forceinline__ void note(int *record, unsigned team) const
    {
        const u64 last = at + (u64)(h + 1) * (n_tiles + BEGIN) - 1;   // the tile that ends it
        const u64 border = more * (size + 1);
        const u64 last_team = last < border ? divide(last, size + 1) : more + divide(last - border, size);
        record[0] = (int)b;
        record[1] = (int)h;
        record[2] = s.count;
        record[3] = (int)((unsigned)last_team - team + 1);     // parts
    }
};

// whether node n of sequence b sees the key; `there` is known
__device__ __forceinline__ bool sees(const AttendArgs &a, unsigned b, const Span &s, int n, unsigned key)
{
    if ((int)key < s.len) return true;
    const unsigned j = key - (unsigned)s.len;
    if (j >= (unsigned)(s.total - s.len)) return false;   // no node, or one behind the table's end
    if (!a.mask) return (int)j <= n;
    return a.mask[b * a.sm[0] + n * a.sm[1] + j] != 0;
}

// zeros for the rows [row0, row0 + m) of nodes that are not there
template <typename T>
__device__ __forceinline__ void absent_rows(const AttendArgs &a, const FastDiv &by_group, unsigned b, unsigned h,
                                            unsigned live, unsigned row0, unsigned m, unsigned t, unsigned threads)
{
    const unsigned rows = a.nodes * by_group.d, dim = a.c.dim;
    const unsigned z0 = max(row0, live), z1 = min(row0 + m, rows);
    if (z0 >= z1) return;
    const unsigned eights = (dim + 7) / 8;
    for (unsigned u = t; u < (z1 - z0) * eights; u += threads) {
        const unsigned r = z0 + u / eights, d = u % eights * 8, node = by_group.div(r), head = h * by_group.d + r - node * by_group.d;
        T *to = static_cast<T *>(a.out) + b * a.so[0] + node * a.so[1] + head * a.so[2] + d;
        if (a.ovec) {
#pragma unroll
            for (int e = 0; e < 8; e += 16 / (int)sizeof(T)) *reinterpret_cast<uint4 *>(to + e) = make_uint4(0, 0, 0, 0);
        } else {
            for (unsigned e = 0; e < 8 && d + e < dim; ++e) to[e] = from_f32<T>(0.0f);
        }
        if (d == 0 && a.lse) a.lse[((size_t)b * a.nodes + node) * a.q_heads + head] = -INFINITY;
    }
}

template <typename T> __device__ __forceinline__ unsigned pack2(float x, float y);
template <> __device__ __forceinline__ unsigned pack2<__nv_bfloat16>(float x, float y)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const unsigned *>(&h);
}
template <> __device__ __forceinline__ unsigned pack2<__half>(float x, float y)
{
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const unsigned *>(&h);
}
template <> __device__ __forceinline__ unsigned pack2<float>(float, float) { return 0; }
template <typename T> __device__ __forceinline__ float2 unpack2(unsigned w);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(unsigned w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(unsigned w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f; }

// Where rows of a CTA's stretch go: to the result or, of a part, to its slot in scratch memory.
template <typename T>
struct RowOut {
    const AttendArgs &a;
    const FastDiv &by_group;
    unsigned b, h, live, row0, m;
    bool part;
    float *slot;

    // entries d to d + 7 (d a multiple of 8) of row r of the tile, its maximum and sum
    __device__ __forceinline__ void put8(unsigned r, unsigned d, const float *x, float top, float sum) const
    {
        const unsigned dim = a.c.dim;
        if (row0 + r >= live || d >= dim) return;
        if (part) {
            float *to = slot + r * dim + d;
            if (dim % 8 == 0) {
                *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4 *>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (d + e < dim) to[e] = x[e];
            }
            if (d == 0) {
                slot[m * dim + 2 * r] = top;
                slot[m * dim + 2 * r + 1] = sum;
            }
            return;
        }
        const unsigned n = by_group.div(row0 + r), head = h * by_group.d + row0 + r - n * by_group.d;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        T *to = static_cast<T *>(a.out) + b * a.so[0] + n * a.so[1] + head * a.so[2] + d;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e] * inv;
        if (a.ovec) {
#pragma unroll
            for (int e = 0; e < 8; e += Pack<T>::N) {
                Pack<T> p;
                p.pack(y + e);
                *reinterpret_cast<uint4 *>(to + e) = p.raw;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (d + e < dim) to[e] = from_f32<T>(y[e]);
        }
        if (d == 0 && a.lse) a.lse[((size_t)b * a.nodes + n) * a.q_heads + head] = lse_of(top, sum);
    }
};

// A row's entries in binary32 on their way out: eights of columns c of row r in shared memory, pieces of 16 bytes turned
// by the row so that a fragment's rows lie in different banks.
__device__ __forceinline__ unsigned out_at(unsigned width, unsigned r, unsigned col)
{
    return r * width + ((((col >> 2) ^ (r & 7u)) << 2) | (col & 3u));
}

// ---- barriers and copies -------------------------------------------------------------------------
__device__ __forceinline__ unsigned smem_u32(const void *p) { return (unsigned)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(unsigned bar, unsigned count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned bar, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(unsigned bar, unsigned parity)
{
    unsigned ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Waits for the phase of the given parity to end; false when it has not after dead[1] milliseconds, or another wait of the CTA
// gave up (dead[0]).
static __device__ __noinline__ bool bar_wait_long(unsigned bar, unsigned parity, volatile unsigned *dead)
{
    u64 began, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(began));
    for (int tries = 0; tries < 1 << 24; ++tries) {
        if (bar_try(bar, parity)) return true;
        if (dead[0]) return false;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (now - began > dead[1] * 1000000ull) break;
    }
    dead[0] = 1;
    return false;
}
__device__ __forceinline__ bool bar_wait(unsigned bar, unsigned parity, volatile unsigned *dead)
{
    return bar_try(bar, parity) || bar_wait_long(bar, parity, dead);
}

// A barrier of the warps that `bar` counts, whose wait ends with the others' (a warp that gave up never comes to it).
struct Meeting {
    unsigned bar, phase;
    __device__ __forceinline__ bool operator()(volatile unsigned *dead)
    {
        __syncwarp();
        if ((threadIdx.x & 31u) == 0) bar_arrive(bar);
        return __all_sync(0xffffffffu, bar_wait(bar, phase++ & 1, dead));
    }
};

// The cache as the copy engine sees it: entries, and slots, heads and pages in the order of their strides.
struct CacheMaps {
    CUtensorMap k, v;
    unsigned char k_at[4], v_at[4];    // the axis (1 .. 3) of slot, head and page
};

__device__ __forceinline__ void load_box(unsigned dst, const CUtensorMap *map, const unsigned char *at, unsigned bar, int d, int slot,
                                         int head, int page)
{
    const int c1 = at[0] == 1 ? slot : at[1] == 1 ? head : page;
    const int c2 = at[0] == 2 ? slot : at[1] == 2 ? head : page;
    const int c3 = at[0] == 3 ? slot : at[1] == 3 ? head : page;
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(map), "r"(d), "r"(c1), "r"(c2), "r"(c3), "r"(bar) : "memory");
}

// One thread of the warp.  (Under a choice like `lane == 0` the compiler does not know that one thread is left: it then
// goes through the active lanes for instructions that take registers of the whole warp, and the addresses of the tensor
// cores' operands came out wrong.)
__device__ __forceinline__ bool chosen()
{
    unsigned one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// What one warp asks for, tile after tile: boxes of 128 bytes by `1 << shift` slots of a page (a power of 2 that
// divides the page), so that a row's 16-byte pieces lie turned by its number modulo 8.  What lies outside the tensor
// (entries past the head's, a page that does not exist) comes as zeros.  The lanes look up the pages of a tile, one
// thread asks for its boxes.
template <int KT>
struct Loader {
    static constexpr int EN = (KT + 31) / 32;
    unsigned shift;            // log2 of the rows of a box
    int *boxes;                // [KT] their pages, in shared memory (16-byte aligned)
    int page[EN];              // of this lane's boxes of the tile that is looked up

    __device__ __forceinline__ void look_up(const AttendArgs &a, unsigned b, const Span &s, unsigned tile)
    {
        const unsigned lane = threadIdx.x & 31u;
#pragma unroll
        for (int e = 0; e < EN; ++e) {
            const unsigned i = lane + 32 * e, key = tile * KT + (i << shift);
            page[e] = (int)a.c.pages;
            if ((i << shift) < KT && key < (unsigned)s.total) page[e] = a.c.table[b * a.c.st + a.c.page.div(key)];
        }
    }

    // hands the boxes to the thread that asks; those without a page as bits of `bad` (null: another warp does)
    __device__ __forceinline__ void hand(const AttendArgs &a, const Span &s, unsigned tile, unsigned *bad, bool tell)
    {
        const unsigned lane = threadIdx.x & 31u;
        bool any = false;
        __syncwarp();          // the boxes of the tile before have been read
#pragma unroll
        for (int e = 0; e < EN; ++e) {
            const unsigned i = lane + 32 * e;
            const bool wrong = (unsigned)page[e] >= a.c.pages && (i << shift) < KT && tile * KT + (i << shift) < (unsigned)s.total;
            const unsigned bits = __ballot_sync(0xffffffffu, wrong);
            if (bad && lane == 0) bad[e] = bits;
            any |= wrong;
            if ((i << shift) < KT) boxes[i] = wrong ? (int)a.c.pages : page[e];
        }
        if (bad && any && tell && a.c.status) atomicOr(a.c.status, PER_DEVFLAG_BAD_INDEX);
        __syncwarp();
    }

    // one array's tile to `to`: [half][KT][128 bytes], at most HN halves.  By the thread that asks.  (Four boxes at a time,
    // so that what one waits for does not keep the next.)
    template <int HN>
    __device__ __forceinline__ void request(const AttendArgs &a, const CUtensorMap *map, const unsigned char *at, unsigned tile, unsigned h,
                                            unsigned to, unsigned halves, unsigned per_half, unsigned bar) const
    {
        bar_expect(bar, halves * KT * 128);
        const unsigned rows = 1u << shift, size = a.c.page.d;
        unsigned slot = tile * KT - a.c.page.div(tile * KT) * size;   // boxes follow one another through a page
        for (unsigned r = 0; r < KT; r += 4 * rows) {
            const int4 four = *reinterpret_cast<const int4 *>(boxes + (r >> shift));
            const int page[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e > 0 && r + e * rows >= KT) break;
#pragma unroll
                for (int half = 0; half < HN; ++half)
                    if (half < (int)halves)
                        load_box(to + half * KT * 128 + (r + e * rows) * 128, map, at, bar, half * per_half, (int)slot, h, page[e]);
                slot += rows;
                if (slot == size) slot = 0;
            }
        }
    }
};

// ---- host --------------------------------------------------------------------------------------
struct Plan {
    unsigned m, row_tiles, teams, grid;
    unsigned share;         // > 0: CTAs (a cluster) that share a sequence's head and rows; 0: the tiles are cut as above
    bool parts;             // a sequence can lie in several CTAs, which the second kernel joins
    u64 bytes;
};

// `shares`: the kernel can take a sequence's head whole; `clusters`: it can join through the shared memory of a cluster's
// CTAs.  Where sequences are short that is quicker than the cut (one kernel, no scratch memory).  Estimated in tiles that a
// CTA works through one after another, a begin counting `begin` and the second kernel 6.  The lengths are not known
// here: the table's width stands for them, and for the cut, which evens ragged lengths out, three quarters of it (their mean
// where they are spread evenly from half of it to all; a table with room to spare leads to the cut).
// Measured, one token of 32 query and 8 key heads of 128 entries: 64 sequences of up to 300 tokens 22.3 us against 24.0
// with the cut, 8 of 2000 17.4 against 18.1; 64 of up to 1500 68 against 57, 16 of 5000 57 against 48.5.
inline Plan plan_of(const AttendArgs &a, unsigned m, unsigned kt, unsigned ctas, unsigned begin, bool shares, bool clusters)
{
    Plan p;
    const u64 rows = (u64)a.nodes * (a.q_heads / a.c.heads);   // at most 2^16
    p.m = m;
    p.row_tiles = (unsigned)((rows + m - 1) / m);
    p.teams = ctas > p.row_tiles ? ctas / p.row_tiles : 1;
    const u64 most = ((u64)a.c.width * a.c.page.d + kt - 1) / kt;   // tiles of a sequence
    const u64 tiles = ((most ? most : 1) + begin) * a.batch * a.c.heads;
    if (p.teams > tiles) p.teams = (unsigned)tiles;
    p.grid = p.teams * p.row_tiles;
    p.share = 0;
    p.parts = most > 1 && p.teams > 1;
    if (p.parts && shares) {
        const u64 units = (u64)a.batch * a.c.heads * p.row_tiles;
        u64 least = (units * (most * 3 / 4 + begin) + ctas - 1) / ctas + 3 + 6;
        for (unsigned n = 1; n <= (clusters ? 8u : 1u); n *= 2) {
            const u64 cost = (units * n + ctas - 1) / ctas * ((most + n - 1) / n + begin);
            if (cost < least && units * n < 1u << 20) {
                least = cost;
                p.share = n;
            }
        }
        if (p.share) {
            p.grid = (unsigned)units * p.share;
            p.parts = false;
        }
    }
    p.bytes = p.parts ? (u64)p.grid * (kRecord * 4 + 2ull * m * (a.c.dim + 2) * 4) : 0;
    return p;
}

// The kernels that take their tiles from the copy engine (k_attend_wide.cu: 16-bit types, heads of up to 128, scale > 0;
// attend_rows.cuh: all).
cudaError_t attend_wide(int type, const AttendArgs &a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes);
cudaError_t attend_rows_f32(const AttendArgs &a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes);
cudaError_t attend_rows_f16(const AttendArgs &a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes);
cudaError_t attend_rows_bf16(const AttendArgs &a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes);
// The maps of a call's cache, whose layout is known to be right.  kt: keys of a tile.
bool make_maps(int type, const AttendArgs &a, unsigned kt, CacheMaps *maps, unsigned *shift);   // k_attend.cu
// joins what several CTAs hold (k_attend.cu)
cudaError_t join_parts(int type, const AttendArgs &a, const Plan &p, const FastDiv &by_group, cudaStream_t st);

}  // namespace attend
}  // namespace gbper
