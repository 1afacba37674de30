// k_attend.cu -- attention of drafted trees over a paged cache.
//
// Mathematics.  A pass over the keys with the running maximum m and sum l of a softmax: for each tile,
// s = scale q k, m' = max(m, max s), p = 2^(s - m'), l = l 2^(m - m') + sum p, o = o 2^(m - m') + p v (scores in units of
// log2).  Parts of a sequence join the same way.  Scores, sums and outputs are binary32; p is rounded
// to the type of v for the matrix instruction, whose products are exact.  binary32 operands are split into a part of
// 11 bits and the rest, and the product of the two rests is dropped.
//
// Work.  The rows of one head of keys are its group of query heads times the nodes; they share every key
// that is read.  A CTA takes up to 64 rows and a stretch of keys, 64 at a time, copied asynchronously
// into a ring of shared memory (the pages are looked up two tiles ahead).  Its four warps share
// the rows where there are many, the keys where there are few, and join at the end.
//
// The stretches: all tiles of all sequences and heads in a row, cut into equal parts, one for each CTA that the
// GPU holds at once (a team of CTAs, where the rows need several).  A part that begins or ends inside a
// sequence leaves its sums in scratch memory, and a second kernel joins them in their order.  So one
// long sequence fills the GPU, and ragged ones leave no SM idle.
#include "ops_internal.cuh"

#include <algorithm>
#include <atomic>

namespace gbper {

namespace {

typedef unsigned long long u64;
constexpr int kThreads = 128;
constexpr int kRecord = 8;             // ints of a CTA's record for the joining kernel
constexpr int kSmemSm = 227 * 1024;

template <typename T, int DP, int WR>
struct Cfg {
    static constexpr int ES = (int)sizeof(T);
    static constexpr int WK = 4 / WR;                       // warps along the keys
    static constexpr int KT = DP * ES > 512 ? 32 : 64;      // keys of a tile
    static constexpr int KW = KT / WK;                      // of them a warp's
    static constexpr int M = 16 * WR;                       // rows of a CTA
    static constexpr int PITCH = DP * ES;                   // bytes of a row in shared memory
    static constexpr int CH = PITCH / 16;
    static constexpr int STAGE = 2 * KT * PITCH;
    static constexpr int QB = M * PITCH;
    static constexpr int ROOM = (STAGE <= 32 * 1024 ? 112 * 1024 : kSmemSm - 1024) - QB - 8 * 1024;
    static constexpr int ST = ROOM / STAGE < 2 ? 2 : ROOM / STAGE > 4 ? 4 : ROOM / STAGE;
    static constexpr int INFO = ST + 1;                     // tiles whose places are kept
    static constexpr int SMEM = ST * STAGE + QB + INFO * KT * 16 + INFO * 8 + 64;
    static constexpr int PER_SM = kSmemSm / (SMEM + 1024);
    static_assert(SMEM <= kSmemSm && PER_SM >= 1, "fits");
    static_assert(WK == 1 || WK * 16 * WR * (DP + 2) * 4 <= ST * STAGE, "the warps' sums lie where the tiles were");
};

// ---- the instructions ------------------------------------------------------------------------
__device__ __forceinline__ unsigned smem_u32(const void *p) { return (unsigned)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void copy16(unsigned dst, const void *src, bool some)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(unsigned *r, unsigned at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(unsigned *r, unsigned at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <typename T> __device__ __forceinline__ void mma16(float *c, const unsigned *a, unsigned b0, unsigned b1);
template <> __device__ __forceinline__ void mma16<__nv_bfloat16>(float *c, const unsigned *a, unsigned b0, unsigned b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <> __device__ __forceinline__ void mma16<__half>(float *c, const unsigned *a, unsigned b0, unsigned b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8(float *c, const unsigned *a, unsigned b0, unsigned b1)
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo, hi of 11 bits (the instruction reads the upper 19 bits of each word)
__device__ __forceinline__ void split(float x, unsigned &hi, unsigned &lo)
{
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
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

// The byte offset of piece c of row r: pieces of 16 bytes are turned so that the rows that an instruction reads
// at once lie in different banks.
template <typename C>
__device__ __forceinline__ unsigned piece(unsigned r, unsigned c)
{
    const unsigned turn = C::ES == 4 ? ((r ^ (r >> 2)) & 3u) << 1 : r & 7u;
    return r * C::PITCH + ((c ^ turn) << 4);
}

// ---- what each CTA does ------------------------------------------------------------------------
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

// (all < 2^45, checked on the host)
__device__ __forceinline__ u64 part_start(u64 t, u64 all, unsigned teams) { return t * all / teams; }

template <typename T, int DP, int WR>
__global__ void __launch_bounds__(kThreads) k_attend(AttendArgs a, unsigned row_tiles, unsigned max_teams, FastDiv by_group)
{
    using C = Cfg<T, DP, WR>;
    constexpr int KT = C::KT, KW = C::KW, WK = C::WK, M = C::M, ST = C::ST;
    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char *tiles = smem;                                   // [ST][keys, values][KT][PITCH]
    unsigned char *qs = smem + ST * C::STAGE;                      // [M][PITCH]
    longlong2 *info = reinterpret_cast<longlong2 *>(qs + C::QB);   // [INFO][KT] element offsets of keys and values
    unsigned *valid = reinterpret_cast<unsigned *>(info + C::INFO * KT);   // [INFO][2] bits: the key is there
    u64 *scan = reinterpret_cast<u64 *>(valid + C::INFO * 2);      // [5]
    const unsigned t = threadIdx.x, lane = t & 31u, warp = t >> 5;
    const unsigned g = lane >> 2, q4 = lane & 3u;                  // row and column pair of a fragment
    const unsigned wr = warp / WK, wk = warp - wr * WK;
    const unsigned cta = blockIdx.x, team = cta / row_tiles, rt = cta - team * row_tiles;
    const unsigned group = by_group.d, heads = a.c.heads, rows = a.nodes * group, row0 = rt * M;
    const unsigned dim = a.c.dim, steps = (dim * C::ES + 31) / 32;  // 32 bytes of a head: a step of the matrix instruction
    const unsigned slot_floats = M * (dim + 2);
    int *record = reinterpret_cast<int *>(a.work) + (size_t)cta * kRecord;
    float *slots = a.work + (size_t)gridDim.x * kRecord + (size_t)cta * 2 * slot_floats;

    pdl_wait();
    pdl_release();

    // where this team's part begins: the tiles of all sequences, summed
    const unsigned per = (a.batch + kThreads - 1) / kThreads;
    const unsigned b0 = min(t * per, a.batch), b1 = min(b0 + per, a.batch);
    u64 mine = 0;
    for (unsigned b = b0; b < b1; ++b) mine += tiles_of<KT>(span(a, b));
    u64 upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const u64 o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    u64 all = 0, before = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < (int)warp) before += scan[w];
        all += scan[w];
    }
    all *= heads;
    before = (before + upto - mine) * heads;                      // tiles in front of this thread's sequences
    const unsigned teams = (unsigned)min((u64)max_teams, all);     // every team has a tile
    u64 pos = team < teams ? part_start(team, all, teams) : all;
    const u64 end = team < teams ? part_start(team + 1, all, teams) : all;
    if (a.work && t == 0) record[3] = 0;
    if (pos >= end) return;
    __syncthreads();
    if (pos >= before && pos < before + mine * heads) {           // one thread's
        unsigned b = b0;
        u64 at = before;
        for (;; ++b) {
            const u64 n = (u64)tiles_of<KT>(span(a, b)) * heads;
            if (pos < at + n) break;
            at += n;
        }
        scan[0] = b;
        scan[1] = at;
    }
    __syncthreads();
    unsigned b = (unsigned)scan[0];
    u64 at = scan[1];                                             // the sequence's first tile

    Span s = span(a, b);
    unsigned n_tiles = tiles_of<KT>(s);
    while (pos < end) {
        if (pos >= at + (u64)n_tiles * heads) {
            at += (u64)n_tiles * heads;
            ++b;
            s = span(a, b);
            n_tiles = tiles_of<KT>(s);
        }
        const unsigned h = (unsigned)((pos - at) / n_tiles);
        const unsigned tile0 = (unsigned)(pos - at - (u64)h * n_tiles);
        const unsigned tile1 = (unsigned)min((u64)n_tiles, tile0 + (end - pos));
        pos += tile1 - tile0;
        if (tile0 == 0 && s.bad && rt == 0 && h == 0 && t == 0 && a.c.status) atomicOr(a.c.status, PER_DEVFLAG_BAD_INDEX);

        // rows of nodes that are not there
        const unsigned live = (unsigned)s.count * group;          // rows that are
        if (tile0 == 0 && row0 + M > live) {
            const unsigned z0 = max(row0, live), z1 = min(row0 + M, rows);
            for (unsigned u = t; z0 < z1 && u < (z1 - z0) * dim; u += kThreads) {
                const unsigned r = z0 + u / dim, d = u % dim, node = by_group.div(r), head = h * group + r - node * group;
                static_cast<T *>(a.out)[b * a.so[0] + node * a.so[1] + head * a.so[2] + d] = from_f32<T>(0.0f);
                if (d == 0 && a.lse) a.lse[((size_t)b * a.nodes + node) * a.q_heads + head] = -INFINITY;
            }
        }
        const bool split_end = tile1 < n_tiles;
        if (split_end && tile0 == 0 && t == 0) {                  // this CTA's last: others go on
            const u64 last = at + (u64)(h + 1) * n_tiles - 1;     // the tile that ends it
            const unsigned last_team = (unsigned)(((last + 1) * teams + all - 1) / all) - 1;
            record[0] = (int)b;
            record[1] = (int)h;
            record[2] = s.count;
            record[3] = (int)(last_team - team + 1);              // parts
        }
        if (row0 >= live) continue;

        // the queries, zero where there is none
        __syncthreads();
        {
            const T *q = static_cast<const T *>(a.q) + b * a.sq[0];
            for (unsigned u = t; u < M * C::CH; u += kThreads) {
                const unsigned r = u / C::CH, c = u % C::CH;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (row0 + r < live) {
                    const unsigned node = by_group.div(row0 + r), head = h * group + row0 + r - node * group;
                    const T *src = q + node * a.sq[1] + head * a.sq[2] + c * (16 / C::ES);
                    if (a.qvec) {
                        if (c * 16 < dim * C::ES) v = *reinterpret_cast<const uint4 *>(src);
                    } else {
                        T e[16 / C::ES];
#pragma unroll
                        for (int i = 0; i < 16 / C::ES; ++i)
                            e[i] = c * (16 / C::ES) + i < dim ? src[i] : from_f32<T>(0.0f);
                        v = *reinterpret_cast<const uint4 *>(e);
                    }
                }
                *reinterpret_cast<uint4 *>(qs + piece<C>(r, c)) = v;
            }
        }
        // where the keys of a tile lie
        auto look_up = [&](unsigned tile) {
            if (t < KT) {
                const unsigned key = tile * KT + t, ring = tile % C::INFO;
                longlong2 w = make_longlong2(0, 0);
                bool there = tile < tile1 && key < (unsigned)s.total;
                if (there) {
                    const unsigned pg = a.c.page.div(key), slot = key - pg * a.c.page.d;
                    const int e = a.c.table[b * a.c.st + pg];
                    there = e >= 0 && (unsigned)e < a.c.pages;
                    if (there) {
                        w.x = e * a.c.sk[0] + slot * a.c.sk[1] + h * a.c.sk[2];
                        w.y = e * a.c.sv[0] + slot * a.c.sv[1] + h * a.c.sv[2];
                    } else if (rt == 0 && h == 0 && a.c.status) {
                        atomicOr(a.c.status, PER_DEVFLAG_BAD_INDEX);
                    }
                }
                const unsigned bits = __ballot_sync(0xffffffffu, there);
                if (lane == 0) valid[ring * 2 + warp] = bits;
                if (!there) w.x = w.y = -1;
                info[ring * KT + t] = w;
            }
        };
        auto request = [&](unsigned tile) {
            if (tile < tile1) {
                unsigned char *ks = tiles + (tile % ST) * C::STAGE, *vs = ks + KT * C::PITCH;
                const longlong2 *in = info + (tile % C::INFO) * KT;
                const unsigned *there = valid + (tile % C::INFO) * 2;
                if (a.c.vec) {
#pragma unroll 4
                    for (unsigned u = t; u < KT * C::CH; u += kThreads) {
                        const unsigned r = u / C::CH, c = u % C::CH;
                        const longlong2 w = in[r];
                        const bool some = (there[r >> 5] >> (r & 31u) & 1u) && c * 16 < dim * C::ES;
                        const char *k = static_cast<const char *>(a.c.k), *v = static_cast<const char *>(a.c.v);
                        copy16(smem_u32(ks + piece<C>(r, c)), some ? k + w.x * C::ES + c * 16 : static_cast<const char *>(a.q), some);
                        copy16(smem_u32(vs + piece<C>(r, c)), some ? v + w.y * C::ES + c * 16 : static_cast<const char *>(a.q), some);
                    }
                } else {
                    for (unsigned u = t; u < KT * C::CH; u += kThreads) {
                        const unsigned r = u / C::CH, c = u % C::CH;
                        const longlong2 w = in[r];
                        const bool some = there[r >> 5] >> (r & 31u) & 1u;
                        const T *k = static_cast<const T *>(a.c.k) + w.x, *v = static_cast<const T *>(a.c.v) + w.y;
                        T e[2][16 / C::ES];
#pragma unroll
                        for (int i = 0; i < 16 / C::ES; ++i) {
                            const unsigned d = c * (16 / C::ES) + i;
                            e[0][i] = some && d < dim ? k[d] : from_f32<T>(0.0f);
                            e[1][i] = some && d < dim ? v[d] : from_f32<T>(0.0f);
                        }
                        *reinterpret_cast<uint4 *>(ks + piece<C>(r, c)) = *reinterpret_cast<const uint4 *>(e[0]);
                        *reinterpret_cast<uint4 *>(vs + piece<C>(r, c)) = *reinterpret_cast<const uint4 *>(e[1]);
                    }
                }
            }
            copy_commit();
        };

        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
        int node[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const unsigned r = row0 + wr * 16 + g + e * 8;
            node[e] = r < live ? (int)by_group.div(r) : -1;       // -1: no such row
        }
        auto sees = [&](int n, unsigned key) {
            if ((int)key < s.len) return true;
            const unsigned j = key - (unsigned)s.len;
            if (j >= (unsigned)s.count) return false;
            if (!a.mask) return (int)j <= n;
            return a.mask[b * a.sm[0] + n * a.sm[1] + j] != 0;
        };

        for (unsigned i = 0; i < ST; ++i) look_up(tile0 + i);
        __syncthreads();
        for (unsigned i = 0; i + 1 < ST; ++i) request(tile0 + i);

        for (unsigned tile = tile0; tile < tile1; ++tile) {
            copy_wait<ST - 2>();
            __syncthreads();                                      // the tile is there, and the one before it is done with
            request(tile + ST - 1);
            look_up(tile + ST);
            unsigned char *ks = tiles + (tile % ST) * C::STAGE, *vs = ks + KT * C::PITCH;
            const unsigned there0 = valid[(tile % C::INFO) * 2], there1 = KT > 32 ? valid[(tile % C::INFO) * 2 + 1] : ~0u;
            const bool nodes_in = (tile + 1) * KT > (unsigned)s.len;
            const bool masked = nodes_in || (there0 & there1) != ~0u;
            const unsigned key0 = wk * KW;                        // the warp's first key of the tile

            // a value that is not finite must reach only the rows that see it
            bool odd = false;
            if (nodes_in) {
                for (unsigned u = t; u < KT * C::CH; u += kThreads) {
                    const unsigned r = u / C::CH;
                    if (tile * KT + r < (unsigned)s.len) continue;
                    Pack<T> p;
                    p.raw = *reinterpret_cast<const uint4 *>(vs + piece<C>(r, u % C::CH));
                    float f[16 / C::ES];
                    p.unpack(f);
                    bool any = false;
#pragma unroll
                    for (int i = 0; i < 16 / C::ES; ++i)
                        if (!(fabsf(f[i]) <= 3.402823466e38f)) {
                            f[i] = 0.0f;
                            any = true;
                        }
                    if (any) {
                        p.pack(f);
                        *reinterpret_cast<uint4 *>(vs + piece<C>(r, u % C::CH)) = p.raw;
                        odd = true;
                    }
                }
                odd = __syncthreads_or(odd);
            }

            float sc[KW / 8][4];
#pragma unroll
            for (int i = 0; i < KW / 8; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.0f;
            if constexpr (C::ES == 2) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    if (k >= (int)steps) break;
                    unsigned qa[4];
                    ldsm4(qa, smem_u32(qs + piece<C>(wr * 16 + (lane & 15u), k * 2 + (lane >> 4))));
#pragma unroll
                    for (int i = 0; i < KW / 16; ++i) {
                        unsigned kb[4];   // keys 0-7 and 8-15, entries 0-7 and 8-15 of each
                        ldsm4(kb, smem_u32(ks + piece<C>(key0 + i * 16 + (lane & 7u) + ((lane >> 4) << 3), k * 2 + ((lane >> 3) & 1u))));
                        mma16<T>(sc[2 * i], qa, kb[0], kb[1]);
                        mma16<T>(sc[2 * i + 1], qa, kb[2], kb[3]);
                    }
                }
            } else {
                // entry 2 c of a step goes with column c of the instruction, 2 c + 1 with column c + 4, on both sides
#pragma unroll
                for (int k = 0; k < DP / 8; ++k) {
                    if (k >= (int)steps) break;
                    unsigned ah[4], al[4];
                    const unsigned r = wr * 16 + g, c = k * 2 + (q4 >> 1), in = (q4 & 1u) * 8;
                    const float2 x = *reinterpret_cast<const float2 *>(qs + piece<C>(r, c) + in);
                    const float2 y = *reinterpret_cast<const float2 *>(qs + piece<C>(r + 8, c) + in);
                    split(x.x, ah[0], al[0]);
                    split(y.x, ah[1], al[1]);
                    split(x.y, ah[2], al[2]);
                    split(y.y, ah[3], al[3]);
#pragma unroll
                    for (int i = 0; i < KW / 8; ++i) {
                        const float2 z = *reinterpret_cast<const float2 *>(ks + piece<C>(key0 + i * 8 + g, c) + in);
                        unsigned h0, l0, h1, l1;
                        split(z.x, h0, l0);
                        split(z.y, h1, l1);
                        mma8(sc[i], al, h0, h1);
                        mma8(sc[i], ah, l0, l1);
                        mma8(sc[i], ah, h0, h1);
                    }
                }
            }

            float up[2] = {top[0], top[1]};
#pragma unroll
            for (int i = 0; i < KW / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[i][e] *= a.c2;
            if (masked) {
#pragma unroll
                for (int i = 0; i < KW / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const unsigned r = key0 + i * 8 + q4 * 2 + (e & 1);
                        const bool there = ((r < 32 ? there0 : there1) >> (r & 31u)) & 1u;
                        if (!there || node[e >> 1] < 0 || !sees(node[e >> 1], tile * KT + r)) sc[i][e] = -INFINITY;
                    }
            }
#pragma unroll
            for (int i = 0; i < KW / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) up[e >> 1] = fmaxf(up[e >> 1], sc[i][e]);
            float keep[2], base[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                up[e] = fmaxf(up[e], __shfl_xor_sync(0xffffffffu, up[e], 1));
                up[e] = fmaxf(up[e], __shfl_xor_sync(0xffffffffu, up[e], 2));
                base[e] = up[e] == -INFINITY ? 0.0f : up[e];      // nothing seen yet: every p is 2^-inf = 0
                keep[e] = ex2(top[e] - base[e]);
                top[e] = up[e];
                sum[e] *= keep[e];
            }
#pragma unroll
            for (int i = 0; i < KW / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[i][e] = ex2(sc[i][e] - base[e >> 1]);
                    sum[e >> 1] += sc[i][e];
                }
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
                o[i][0] *= keep[0];
                o[i][1] *= keep[0];
                o[i][2] *= keep[1];
                o[i][3] *= keep[1];
            }
            if constexpr (C::ES == 2) {
#pragma unroll
                for (int k = 0; k < KW / 16; ++k) {
                    const unsigned pa[4] = {pack2<T>(sc[2 * k][0], sc[2 * k][1]), pack2<T>(sc[2 * k][2], sc[2 * k][3]),
                                            pack2<T>(sc[2 * k + 1][0], sc[2 * k + 1][1]), pack2<T>(sc[2 * k + 1][2], sc[2 * k + 1][3])};
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i) {
                        if (i >= (int)steps) break;
                        unsigned vb[4];   // keys 0-7 and 8-15 of entries 0-7, then of entries 8-15
                        ldsm4t(vb, smem_u32(vs + piece<C>(key0 + k * 16 + (lane & 15u), i * 2 + (lane >> 4))));
                        mma16<T>(o[2 * i], pa, vb[0], vb[1]);
                        mma16<T>(o[2 * i + 1], pa, vb[2], vb[3]);
                    }
                }
            } else {
                // key 2 c goes with column c of the instruction, 2 c + 1 with column c + 4: the scores lie so already
#pragma unroll
                for (int k = 0; k < KW / 8; ++k) {
                    unsigned ph[4], pl[4];
                    split(sc[k][0], ph[0], pl[0]);
                    split(sc[k][2], ph[1], pl[1]);
                    split(sc[k][1], ph[2], pl[2]);
                    split(sc[k][3], ph[3], pl[3]);
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i) {
                        if (i >= (int)steps) break;
                        const unsigned r = key0 + k * 8 + q4 * 2, c = i * 2 + (g >> 2), in = (g & 3u) * 4;
                        const float x = *reinterpret_cast<const float *>(vs + piece<C>(r, c) + in);
                        const float y = *reinterpret_cast<const float *>(vs + piece<C>(r + 1, c) + in);
                        unsigned h0, l0, h1, l1;
                        split(x, h0, l0);
                        split(y, h1, l1);
                        mma8(o[i], pl, h0, h1);
                        mma8(o[i], ph, l0, l1);
                        mma8(o[i], ph, h0, h1);
                    }
                }
            }
            if (odd) {   // what was taken out, for the rows that see it (rare: nothing here is fast)
                for (unsigned r = key0; r < key0 + KW; ++r) {
                    const unsigned key = tile * KT + r;
                    if ((int)key < s.len || !(((r < 32 ? there0 : there1) >> (r & 31u)) & 1u)) continue;
                    const T *v = static_cast<const T *>(a.c.v) + info[(tile % C::INFO) * KT + r].y;
                    const bool see[2] = {node[0] >= 0 && sees(node[0], key), node[1] >= 0 && sees(node[1], key)};
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const unsigned d = i * 8 + q4 * 2 + (e & 1);
                            if (d >= dim || !see[e >> 1]) continue;
                            const float x = to_f32(v[d]);
                            if (!(fabsf(x) <= 3.402823466e38f)) o[i][e] += x;
                        }
                }
            }
        }
        copy_wait<0>();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
            sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
        }

        // out: to the result, or (a part) to this CTA's slot
        const bool part = tile0 != 0 || split_end;
        float *slot = slots + (tile0 != 0 ? 0 : slot_floats);
        auto emit = [&](unsigned r, unsigned d, float x, float y, float m, float l) {   // two entries of row r
            if (row0 + r >= live) return;
            if (part) {
                float *to = slot + r * dim + d;
                if (d < dim) to[0] = x;
                if (d + 1 < dim) to[1] = y;
                if (d == 0) {
                    slot[M * dim + 2 * r] = m;
                    slot[M * dim + 2 * r + 1] = l;
                }
                return;
            }
            const unsigned n = by_group.div(row0 + r), head = h * group + row0 + r - n * group;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            T *to = static_cast<T *>(a.out) + b * a.so[0] + n * a.so[1] + head * a.so[2] + d;
            if (C::ES == 2 && a.opair) {
                if (d < dim) *reinterpret_cast<unsigned *>(to) = pack2<T>(x * inv, y * inv);
            } else {
                if (d < dim) to[0] = from_f32<T>(x * inv);
                if (d + 1 < dim) to[1] = from_f32<T>(y * inv);
            }
            if (d == 0 && a.lse)
                a.lse[((size_t)b * a.nodes + n) * a.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        };
        if constexpr (WK == 1) {
#pragma unroll
            for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    emit(wr * 16 + g + e * 8, i * 8 + q4 * 2, o[i][2 * e], o[i][2 * e + 1], top[e], sum[e]);
        } else {
            __syncthreads();                                      // the tiles are done with
            float *os = reinterpret_cast<float *>(tiles);         // [WK][M][DP], then m and l [WK][M][2]
            float *ml = os + WK * M * DP;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const unsigned r = wr * 16 + g + e * 8;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i)
                    *reinterpret_cast<float2 *>(os + (wk * M + r) * DP + i * 8 + q4 * 2) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
                if (q4 == 0) {
                    ml[(wk * M + r) * 2] = top[e];
                    ml[(wk * M + r) * 2 + 1] = sum[e];
                }
            }
            __syncthreads();
            for (unsigned u = t; u < M * (DP / 2); u += kThreads) {
                const unsigned r = u / (DP / 2), d = u % (DP / 2) * 2;
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < WK; ++w) m = fmaxf(m, ml[(w * M + r) * 2]);
                const float base = m == -INFINITY ? 0.0f : m;
                float x = 0.0f, y = 0.0f, l = 0.0f;
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                    const float f = ex2(ml[(w * M + r) * 2] - base);
                    const float2 z = *reinterpret_cast<const float2 *>(os + (w * M + r) * DP + d);
                    x += f * z.x;
                    y += f * z.y;
                    l += f * ml[(w * M + r) * 2 + 1];
                }
                emit(r, d, x, y, m, l);
            }
        }
    }
}

// Joins the parts of what lies in several CTAs: each CTA that begins such a stretch left a record.  A warp
// takes a row, a lane four entries (and further ones of heads above 128).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_attend_join(AttendArgs a, unsigned row_tiles, unsigned m_rows, FastDiv by_group)
{
    const unsigned cta = blockIdx.x, team = cta / row_tiles, rt = cta - team * row_tiles;
    pdl_wait();
    pdl_release();
    const int *record = reinterpret_cast<const int *>(a.work) + (size_t)cta * kRecord;
    const int parts = record[3];
    if (parts == 0) return;
    const unsigned b = (unsigned)record[0], h = (unsigned)record[1], count = (unsigned)record[2];
    const unsigned group = by_group.d, live = count * group, dim = a.c.dim, slot_floats = m_rows * (dim + 2);
    const unsigned r = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31u, row = rt * m_rows + r;
    if (r >= m_rows || row >= live) return;
    const float *slots = a.work + (size_t)gridDim.x * kRecord;
    auto slot = [&](int i) {   // the first part lies in its CTA's second slot, the others in their first
        return slots + ((size_t)((team + i) * row_tiles + rt) * 2 + (i == 0)) * slot_floats;
    };
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, slot(i)[m_rows * dim + 2 * r]);
#pragma unroll
    for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float base = m == -INFINITY ? 0.0f : m;
    constexpr int E = 8;       // 32 lanes x 8 entries
    float acc[E] = {}, l = 0.0f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float *p = slot(i);
        const float f = ex2(p[m_rows * dim + 2 * r] - base);
        l += f * p[m_rows * dim + 2 * r + 1];
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e * 32 + lane < dim) acc[e] += f * p[r * dim + e * 32 + lane];
    }
    const unsigned node = by_group.div(row), head = h * group + row - node * group;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T *to = static_cast<T *>(a.out) + b * a.so[0] + node * a.so[1] + head * a.so[2];
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e * 32 + lane < dim) to[e * 32 + lane] = from_f32<T>(acc[e] * inv);
    if (lane == 0 && a.lse)
        a.lse[((size_t)b * a.nodes + node) * a.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// ---- launches ----------------------------------------------------------------------------------
struct Plan {
    unsigned m, row_tiles, teams, grid;
    bool parts;             // a sequence can lie in several CTAs
    u64 bytes;
};

template <typename C>
Plan plan_of(const AttendArgs &a, unsigned sms)
{
    Plan p;
    const u64 rows = (u64)a.nodes * (a.q_heads / a.c.heads);      // at most 2^16
    p.m = C::M;
    p.row_tiles = (unsigned)((rows + C::M - 1) / C::M);
    p.teams = std::max(1u, sms * C::PER_SM / p.row_tiles);
    const u64 most = ((u64)a.c.width * a.c.page.d + C::KT - 1) / C::KT;   // tiles of a sequence
    const u64 tiles = std::max<u64>(most, 1) * a.batch * a.c.heads;
    p.teams = (unsigned)std::min<u64>(p.teams, tiles);
    p.grid = p.teams * p.row_tiles;
    p.parts = most > 1 && p.teams > 1;
    p.bytes = p.parts ? (u64)p.grid * (kRecord * 4 + 2ull * C::M * (a.c.dim + 2) * 4) : 0;
    return p;
}

template <typename T, int DP, int WR>
cudaError_t attend(AttendArgs a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    using C = Cfg<T, DP, WR>;
    const Plan p = plan_of<C>(a, (unsigned)dev.sms);
    if (bytes) {
        *bytes = p.bytes;
        return cudaSuccess;
    }
    static std::atomic<bool> done[64];   // (two threads may both set the attribute, to the same value)
    if (!done[dev.device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(k_attend<T, DP, WR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        done[dev.device].store(true, std::memory_order_release);
    }
    if (!p.parts) a.work = nullptr;
    FastDiv by_group;
    by_group.set(a.q_heads / a.c.heads);
    cudaError_t e = launch_clusters(k_attend<T, DP, WR>, p.grid, kThreads, 1, C::SMEM, st, a, p.row_tiles, p.teams, by_group);
    if (e != cudaSuccess || !p.parts) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid, (p.m + 3) / 4);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attend_join<T>, a, p.row_tiles, p.m, by_group);
}

template <typename T, int DP>
cudaError_t attend_d(const AttendArgs &a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    const unsigned rows = a.nodes * (a.q_heads / a.c.heads);
    if (rows <= 16) return attend<T, DP, 1>(a, dev, st, bytes);
    if (rows <= 32) return attend<T, DP, 2>(a, dev, st, bytes);
    return attend<T, DP, 4>(a, dev, st, bytes);
}

template <typename T>
cudaError_t attend_t(const AttendArgs &a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    if (a.c.dim <= 64) return attend_d<T, 64>(a, dev, st, bytes);
    if (a.c.dim <= 128) return attend_d<T, 128>(a, dev, st, bytes);
    return attend_d<T, 256>(a, dev, st, bytes);
}

cudaError_t attend_any(int type, const AttendArgs &a, cudaStream_t st, u64 *bytes)
{
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    if (type == PER_TYPE_F32) return attend_t<float>(a, dev, st, bytes);
    if (type == PER_TYPE_F16) return attend_t<__half>(a, dev, st, bytes);
    return attend_t<__nv_bfloat16>(a, dev, st, bytes);
}

}  // namespace

cudaError_t launch_attend(int type, const AttendArgs &a, cudaStream_t st) { return attend_any(type, a, st, nullptr); }

cudaError_t attend_work(int type, const AttendArgs &a, unsigned long long *bytes)
{
    return attend_any(type, a, nullptr, bytes);
}

}  // namespace gbper
