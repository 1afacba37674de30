// attend_rows.cuh -- attention over a paged cache for few rows: one warp asks the copy engine for tiles of keys
// and values, four warps work on them.
//
// The rows of a head of keys (its query heads times the nodes) share every key that is read, so that HBM bounds
// the kernel while they are few.  A CTA takes 16, 32 or 64 rows.  Its four warps share the rows where there are
// many, the keys of a tile where there are few, and then join through shared memory at the end of a
// stretch.  Tiles of 32 KB (64 KB of large heads) lie in a ring of barriers: a warp that is done with one
// never waits for the others, and the copies of the next stretch begin while this one is joined.
//
// Measured (GB300): 64 sequences of up to 5000 tokens, 32 query heads on 8 of 128 entries, bf16, pages of 16 151 us,
// 6.12 TB/s (92% of the copy rate); one of 262145 tokens, 8 nodes, 32 rows a head 176 us (91%); one token over 1023
// 9.3 us.  binary32: 5 trees of 13 nodes, up to 3001 tokens, 12 heads of 80 entries 49 us (29%), the first ones decoding 491 us
// (60%).  Its products, three for one, are not the limit (42 TFLOP/s of them in the former): a warp has 8 keys of a tile, so
// that operands are read from shared memory for three products at a time, in one short chain.  Pages that hold no 16
// slots in a row come as smaller boxes, of which the copy engine takes one in about 64 cycles.
#pragma once

#include "attend_mma.cuh"

#include <algorithm>
#include <atomic>

namespace gbper {
namespace attend {
namespace {

constexpr unsigned kBegin = 3;             // tiles that a sequence's begin and end are worth
constexpr int kWarps = 4;                  // of them that compute
constexpr int kThreads = kWarps * 32 + 64;   // and a warp that asks for keys, one for values

// What lies behind the tiles and the queries: barriers, and what goes from warp to warp.
template <int KT, int ML, int ST>
struct Tail {
    u64 full[2 * ST], empty[ST], meet;   // full: keys, then values
    u64 scan[kThreads / 32];
    unsigned bad[ST][KT / 32];
    alignas(8) float ml[ML][2];   // maxima and sums that the warps hand over
    alignas(16) int boxes[2][KT];
    unsigned asked[2];         // tiles that the warps have asked for in all
    unsigned dead[2], odd;     // whether a wait gave up, and their limit; odd: the number of the last tile that something was taken out of
};

template <typename T, int DP, int WR>
struct Cfg {
    static constexpr int ES = (int)sizeof(T);
    static constexpr int WK = kWarps / WR;                        // warps along the keys
    static constexpr int M = 16 * WR;                             // rows of a CTA
    static constexpr int KT = ES == 4 ? (DP >= 128 ? 32 : 64) : DP >= 128 ? 64 : 128;
    static constexpr int KW = KT / WK;                            // keys of a warp
    static constexpr int PER_HALF = 128 / ES;
    static constexpr int STAGE = 2 * KT * DP * ES;
    static constexpr int JOIN = WK == 4 ? 2 * 16 * DP * 4 : WK == 2 ? M * DP * 4 : 0;   // what the warps hand over
    static constexpr int QB = M * DP * ES * (ES == 4 ? 2 : 1);                          // the queries lie there before
    static constexpr int AREA = QB > JOIN ? QB : JOIN;
    static constexpr int TAIL = KT == 128 || WR == 4 ? 2048 : 1024;
    static constexpr int HALF_SM = 228 * 1024 / 2 - 1024;
    static constexpr int WHOLE_SM = 227 * 1024;
    static constexpr int PER_SM = (HALF_SM - AREA - TAIL) / STAGE >= (ES == 4 ? 2 : 3) ? 2 : 1;
    static constexpr int FIT = ((PER_SM == 2 ? HALF_SM : WHOLE_SM) - AREA - TAIL) / STAGE;
    static constexpr int ST = FIT > 6 ? 6 : FIT;
    static constexpr int SMEM = ST * STAGE + AREA + TAIL;
    typedef Tail<KT, WK == 1 ? M : 32, ST> End;
    static_assert(ST >= 2 && sizeof(End) <= TAIL, "fits");
    static_assert(ES == 4 || KW % 16 == 0, "whole steps of the matrix instruction");
};

// two and four words at the same place of the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ float2 far2(const float *p, unsigned rank)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cluster_smem_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float4 far4(const float *p, unsigned rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_smem_addr(p, rank)) : "memory");
    return v;
}

template <typename T, int DP, int WR>
__global__ void __launch_bounds__(kThreads, Cfg<T, DP, WR>::PER_SM)
k_attend_rows(const __grid_constant__ CacheMaps maps, AttendArgs a, unsigned row_tiles, unsigned max_teams, FastDiv by_group, unsigned shift, unsigned share)
{
    using C = Cfg<T, DP, WR>;
    constexpr int KT = C::KT, KW = C::KW, WK = C::WK, M = C::M, ST = C::ST, ES = C::ES;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *area = smem + ST * C::STAGE;
    typename C::End &tail = *reinterpret_cast<typename C::End *>(area + C::AREA);
    volatile unsigned *dead = tail.dead;
    const unsigned t = threadIdx.x, lane = t & 31u, warp = t >> 5;
    const unsigned cta = blockIdx.x, unit = share ? cta / share : cta, team = unit / row_tiles, rt = unit - team * row_tiles;
    const unsigned rank = share ? cta - unit * share : 0;         // in a cluster that shares a sequence's head and rows
    const unsigned group = by_group.d, row0 = rt * M, dim = a.c.dim;
    const unsigned halves = (dim * ES + 127) / 128;
    const unsigned full = smem_u32(tail.full), empty = smem_u32(tail.empty);

    if (t == 0) {
        for (int i = 0; i < ST; ++i) {
            bar_init(full + 8 * i, 1 + (a.withhold == kKeys));
            bar_init(full + 8 * (ST + i), 1 + (a.withhold == kValues));
            bar_init(empty + 8 * i, kWarps + (a.withhold == kRelease));
        }
        bar_init(smem_u32(&tail.meet), kWarps + (a.withhold == kMeet));
        tail.dead[0] = 0;
        tail.dead[1] = a.wait_ms;
        tail.odd = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pdl_wait();
    pdl_release();
    int *record = reinterpret_cast<int *>(a.work) + (size_t)cta * kRecord;
    if (a.work && t == 0) record[3] = 0;
    Walk<KT, kBegin> w;
    if (share) {
        __syncthreads();
        w.one(a, team / a.c.heads, team % a.c.heads, rank, share);
    } else if (!w.template begin<kThreads>(a, team, max_teams, tail.scan)) {
        return;
    }
    unsigned turns = 0;
    auto next = [&] { return share ? turns++ == 0 : w.next(a); };
    unsigned st = 0, phase = 0;

    if (warp >= kWarps) {   // the warps that ask for tiles: a box takes a thread some 150 cycles
        const bool val = warp > kWarps;
        const unsigned mine = full + (val ? 8 * ST : 0), at = val ? KT * DP * ES : 0;
        const CUtensorMap *map = val ? &maps.v : &maps.k;
        const unsigned char *axes = val ? maps.v_at : maps.k_at;
        Loader<KT> load;
        load.shift = shift;
        load.boxes = tail.boxes[val];
        unsigned asked = 0;
        bool ok = true;
        const bool one = chosen();
        while (ok && next()) {
            if (row0 >= (unsigned)w.s.count * group) continue;
            load.look_up(a, w.b, w.s, w.tile0);
            for (unsigned tile = w.tile0; tile < w.tile1; ++tile) {
                if (asked >= (unsigned)ST) ok = __all_sync(0xffffffffu, bar_wait(empty + 8 * st, phase ^ 1, dead));
                if (!ok) break;
                load.hand(a, w.s, tile, val ? nullptr : tail.bad[st], rt == 0 && w.h == 0);
                if (one)
                    load.template request<DP * ES / 128>(a, map, axes, tile, w.h, smem_u32(smem + st * C::STAGE) + at, halves, C::PER_HALF,
                                                         mine + 8 * st);
                ++asked;
                if (++st == ST) {
                    st = 0;
                    phase ^= 1;
                }
                if (tile + 1 < w.tile1) load.look_up(a, w.b, w.s, tile + 1);
            }
        }
        if (lane == 0) tail.asked[val] = asked;
    } else {
        const unsigned g = lane >> 2, q4 = lane & 3u;                // row and column pair of a fragment
        const unsigned wr = warp / WK, wk = warp - wr * WK, key0 = wk * KW;
        const unsigned slot_floats = M * (dim + 2);
        float *slots = a.work + (size_t)gridDim.x * kRecord + (size_t)cta * 2 * slot_floats;
        Meeting meet{smem_u32(&tail.meet), 0};
        unsigned tiles_done = 0;
        bool ok = true;
        while (ok && next()) {
            const Span &s = w.s;
            const unsigned b = w.b, h = w.h;
            const bool begins = w.tile0 == 0 && rank == 0;
            if (begins && s.bad && rt == 0 && h == 0 && t == 0 && a.c.status) atomicOr(a.c.status, PER_DEVFLAG_BAD_INDEX);
            const unsigned live = (unsigned)s.count * group;         // rows of nodes that are there
            if (begins) absent_rows<T>(a, by_group, b, h, live, row0, M, t, kWarps * 32);
            if (row0 >= live) {
                if (!share && begins && w.tile1 < w.n_tiles && t == 0) w.note(record, team);
                continue;
            }

            // the queries, zero where there is none
            if (!(ok = meet(dead))) break;
            {
                // eight requests at a time, so that their latencies overlap
                constexpr unsigned CH = DP * ES / 16, ALL = M * CH / (kWarps * 32), EACH = ALL < 8 ? ALL : 8;
                const T *q = static_cast<const T *>(a.q) + b * a.sq[0];
#pragma unroll 1
                for (unsigned u0 = 0; u0 < ALL; u0 += EACH) {
                    uint4 v[EACH];
#pragma unroll
                    for (unsigned i = 0; i < EACH; ++i) {
                        const unsigned u = t + (u0 + i) * kWarps * 32, r = u / CH, c = u % CH;
                        const bool some = row0 + r < live;
                        const unsigned node = by_group.div(row0 + r), head = h * group + row0 + r - node * group;
                        const T *src = some ? q + node * a.sq[1] + head * a.sq[2] : q;
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (!a.qvec) v[i] = entries<T>(src, c, dim, some);
                        else if (some && c * 16 < dim * ES) v[i] = *reinterpret_cast<const uint4 *>(src + c * (16 / ES));
                    }
#pragma unroll
                    for (unsigned i = 0; i < EACH; ++i) {
                        const unsigned u = t + (u0 + i) * kWarps * 32, r = u / CH, c = u % CH;
                        if constexpr (ES == 4) {   // both parts of each
                            uint4 lo;
                            split(__uint_as_float(v[i].x), v[i].x, lo.x);
                            split(__uint_as_float(v[i].y), v[i].y, lo.y);
                            split(__uint_as_float(v[i].z), v[i].z, lo.z);
                            split(__uint_as_float(v[i].w), v[i].w, lo.w);
                            *reinterpret_cast<uint4 *>(area + M * DP * ES + piece(M, r, c)) = lo;
                        }
                        *reinterpret_cast<uint4 *>(area + piece(M, r, c)) = v[i];
                    }
                }
            }
            float o[DP / 8][4];
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
            float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
            int node[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const unsigned r = row0 + wr * 16 + g + e * 8;
                node[e] = r < live ? (int)by_group.div(r) : -1;      // -1: no such row
            }
            if (!(ok = meet(dead))) break;

            for (unsigned tile = w.tile0; tile < w.tile1; ++tile) {
                ok = __all_sync(0xffffffffu, bar_wait(full + 8 * st, phase, dead));
                if (!ok) break;
                unsigned char *ks = smem + st * C::STAGE, *vs = ks + KT * DP * ES;
                const bool tail_in = (tile + 1) * KT > (unsigned)s.len;   // nodes, or the end
                unsigned wrong = 0;
#pragma unroll
                for (int e = 0; e < Loader<KT>::EN; ++e) wrong |= tail.bad[st][e];

                // what stale slots hold is taken out of the values, and what is not finite in a node's: it must
                // reach only the rows that see it
                bool odd = false;
                ++tiles_done;
                if (tail_in) {
                    if (!(ok = __all_sync(0xffffffffu, bar_wait(full + 8 * (ST + st), phase, dead)))) break;
                    odd = clean<T>(vs, KT, tile * KT, s, halves * 8, t, kWarps * 32);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the next copy comes after these stores
                    if (odd) tail.odd = tiles_done;
                    if (!(ok = meet(dead))) break;
                    odd = *(volatile unsigned *)&tail.odd >= tiles_done;   // (a warp ahead may have written the next tile's)
                }

                float sc[KW / 8][4];
                scores<T, DP, KW>(sc, area, M, wr * 16, ks, KT, key0, halves);
#pragma unroll
                for (int i = 0; i < KW / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[i][e] *= a.c2;
                if (tail_in || wrong)
                    hide<KW>(sc, a, b, s, node, tile * KT, key0, [&](unsigned r) {
                        return !wrong || !((tail.bad[st][r >> shift >> 5] >> (r >> shift & 31u)) & 1u);
                    });
                if constexpr (ES == 4) once_more<KW>(sc, a, b, h, group, node, row0 + wr * 16 + g, ks, KT, key0);
                soften<T, DP, KW>(sc, top, sum, o);
                if (!tail_in && !(ok = __all_sync(0xffffffffu, bar_wait(full + 8 * (ST + st), phase, dead)))) break;
                values<T, DP, KW, WR == 1>(o, sc, vs, KT, key0, halves);
                if (odd)
                    for (unsigned r = key0; r < key0 + KW; ++r) {
                        const unsigned key = tile * KT + r, box = r >> shift;
                        if ((int)key < s.len || key >= (unsigned)s.total || ((tail.bad[st][box >> 5] >> (box & 31u)) & 1u)) continue;
                        const unsigned pg = a.c.page.div(key);
                        give_back<T, DP>(a, b, s, node, key,
                                         static_cast<const T *>(a.c.v) + a.c.table[b * a.c.st + pg] * a.c.sv[0] +
                                             (key - pg * a.c.page.d) * a.c.sv[1] + h * a.c.sv[2], o);
                    }
                __syncwarp();
                if (lane == 0) bar_arrive(empty + 8 * st);
                if (++st == ST) {
                    st = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
                sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
                top[e] = below<T>(top[e]);      // from here on what the sums refer to
            }

            // the warps that share rows join: the upper two hand their sums to the lower two; what is left lies in one
            // or two areas of [row][entry], and all warps write it out
            constexpr int AREAS = WK == 4 ? 2 : 1;
            constexpr int WIDE = WK == 1 && ES == 2 ? DP / 2 : DP;        // entries that an area holds at once
            float *sums = reinterpret_cast<float *>(area);
            if (!(ok = meet(dead))) break;                              // the queries are done with
            if (!share && begins && w.tile1 < w.n_tiles && t == 0) w.note(record, team);
            if constexpr (WK > 1) {
                const unsigned i = WK == 4 ? wk & 1u : wr;              // the area that a pair shares
                if (wk >= (unsigned)WK / 2) {
                    float *to = sums + i * 16 * DP;
#pragma unroll
                    for (int k = 0; k < DP / 8; ++k)
                        *reinterpret_cast<float4 *>(to + (k * 32 + lane) * 4) = make_float4(o[k][0], o[k][1], o[k][2], o[k][3]);
                    if (q4 == 0) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            tail.ml[i * 16 + g + e * 8][0] = top[e];
                            tail.ml[i * 16 + g + e * 8][1] = sum[e];
                        }
                    }
                }
                if (!(ok = meet(dead))) break;
                if (wk < (unsigned)WK / 2) {
                    const float *from = sums + i * 16 * DP;
                    float mine[2], other[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m = tail.ml[i * 16 + g + e * 8][0], l = tail.ml[i * 16 + g + e * 8][1];
                        const float up = fmaxf(top[e], m), base = up == -INFINITY ? 0.0f : up;
                        mine[e] = ex2(top[e] - base);
                        other[e] = ex2(m - base);
                        sum[e] = sum[e] * mine[e] + l * other[e];
                        top[e] = up;
                    }
#pragma unroll
                    for (int k = 0; k < DP / 8; ++k) {
                        const float4 x = *reinterpret_cast<const float4 *>(from + (k * 32 + lane) * 4);
                        o[k][0] = o[k][0] * mine[0] + x.x * other[0];
                        o[k][1] = o[k][1] * mine[0] + x.y * other[0];
                        o[k][2] = o[k][2] * mine[1] + x.z * other[1];
                        o[k][3] = o[k][3] * mine[1] + x.w * other[1];
                    }
                    __syncwarp();
                }
            }
            const RowOut<T> out{a, by_group, b, h, live, row0, M, !share && w.part(), slots + (w.tile0 != 0 ? 0 : slot_floats)};
#pragma unroll
            for (int d0 = 0; d0 < DP; d0 += WIDE) {
                if (d0 > 0 && !(ok = meet(dead))) break;
                if (WK == 1 || wk < (unsigned)WK / 2) {
                    const unsigned i = WK == 4 ? wk * 16 : wr * 16;         // the first row of this warp's in the areas
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int k = d0 / 8; k < (d0 + WIDE) / 8; ++k)
                            *reinterpret_cast<float2 *>(sums + out_at(WIDE, i + g + e * 8, k * 8 - d0 + q4 * 2)) =
                                make_float2(o[k][2 * e], o[k][2 * e + 1]);
                        if (q4 == 0) {
                            tail.ml[i + g + e * 8][0] = top[e];
                            tail.ml[i + g + e * 8][1] = sum[e];
                        }
                    }
                }
                if (share > 1) break;                                   // the cluster goes on below
                if (!(ok = meet(dead))) break;
                for (unsigned u = t; u < M * (WIDE / 8); u += kWarps * 32) {
                    const unsigned r = u / (WIDE / 8), c = u % (WIDE / 8) * 8;
                    if (row0 + r >= live || d0 + c >= dim) continue;
                    float m = tail.ml[r][0], l = tail.ml[r][1], f[2] = {1.0f, 0.0f};
                    if (AREAS == 2) {
                        const float m1 = tail.ml[16 + r][0], up = fmaxf(m, m1), base = up == -INFINITY ? 0.0f : up;
                        f[0] = ex2(m - base);
                        f[1] = ex2(m1 - base);
                        l = l * f[0] + tail.ml[16 + r][1] * f[1];
                        m = up;
                    }
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 y = *reinterpret_cast<const float4 *>(sums + out_at(WIDE, r, c + e));
                        x[e] = y.x, x[e + 1] = y.y, x[e + 2] = y.z, x[e + 3] = y.w;
                        if (AREAS == 2) {
                            const float4 z = *reinterpret_cast<const float4 *>(sums + out_at(WIDE, 16 + r, c + e));
                            x[e] = x[e] * f[0] + z.x * f[1];
                            x[e + 1] = x[e + 1] * f[0] + z.y * f[1];
                            x[e + 2] = x[e + 2] * f[0] + z.z * f[1];
                            x[e + 3] = x[e + 3] * f[0] + z.w * f[1];
                        }
                    }
                    out.put8(r, d0 + c, x, m, l);
                }
            }
        }
        if (!ok && lane == 0 && a.c.status) atomicOr(a.c.status, PER_DEVFLAG_TIMEOUT);
    }
    __syncthreads();
    if (tail.dead[0]) {   // a wait gave up, be it the last one: nobody leaves before the copies under way have landed
        if (warp >= kWarps) {
            const unsigned asked = tail.asked[warp - kWarps], mine = full + (warp - kWarps) * 8 * ST;
            for (unsigned i = asked > (unsigned)ST ? asked - ST : 0; i < asked; ++i) {
                unsigned none[2] = {0, a.wait_ms};
                bar_wait(mine + 8 * (i % ST), i / ST & 1, none);
            }
        }
        __syncthreads();
    }
    if constexpr (WK > 1) {
        if (share > 1) {   // each CTA joins a part of the rows from all of them
            cluster_sync_all();
            const unsigned live = (unsigned)w.s.count * group;
            if (warp < kWarps && row0 < live) {
                constexpr unsigned AREAS = WK == 4 ? 2 : 1;
                const RowOut<T> out{a, by_group, w.b, w.h, live, row0, M, false, nullptr};
                const float *sums = reinterpret_cast<const float *>(area);
                for (unsigned u = rank * kWarps * 32 + t; u < M * (DP / 8); u += share * kWarps * 32) {
                    const unsigned r = u / (DP / 8), c = u % (DP / 8) * 8;
                    if (row0 + r >= live || c >= dim) continue;
                    float m = -INFINITY, l = 0.0f, x[8] = {};
                    for (unsigned i = 0; i < share; ++i)
#pragma unroll
                        for (unsigned k = 0; k < AREAS; ++k) m = fmaxf(m, far2(&tail.ml[k * 16 + r][0], i).x);
                    const float base = m == -INFINITY ? 0.0f : m;
                    for (unsigned i = 0; i < share; ++i)
#pragma unroll
                        for (unsigned k = 0; k < AREAS; ++k) {
                            const float2 z = far2(&tail.ml[k * 16 + r][0], i);
                            const float f = ex2(z.x - base);
                            l += f * z.y;
                            const float4 p = far4(sums + out_at(DP, k * 16 + r, c), i), q = far4(sums + out_at(DP, k * 16 + r, c + 4), i);
                            x[0] += f * p.x, x[1] += f * p.y, x[2] += f * p.z, x[3] += f * p.w;
                            x[4] += f * q.x, x[5] += f * q.y, x[6] += f * q.z, x[7] += f * q.w;
                        }
                    out.put8(r, c, x, m, l);
                }
            }
            cluster_sync_all();   // nobody leaves before its sums are read
        }
    }
}

template <typename T, int DP, int WR>
cudaError_t rows(AttendArgs a, int type, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    using C = Cfg<T, DP, WR>;
    const Plan p = plan_of(a, C::M, C::KT, (unsigned)dev.sms * C::PER_SM, kBegin, true, C::WK > 1);
    if (bytes) {
        *bytes = p.parts ? p.bytes : 0;
        return cudaSuccess;
    }
    CacheMaps maps;
    unsigned shift;
    if (!make_maps(type, a, C::KT, &maps, &shift)) return cudaErrorInvalidValue;
    static std::atomic<bool> done[64];   // (two threads may both set the attribute, to the same value)
    if (!done[dev.device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(k_attend_rows<T, DP, WR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        done[dev.device].store(true, std::memory_order_release);
    }
    if (!p.parts) a.work = nullptr;
    FastDiv by_group;
    by_group.set(a.q_heads / a.c.heads);
    const cudaError_t e = launch_clusters(k_attend_rows<T, DP, WR>, p.grid, kThreads, std::max(p.share, 1u), C::SMEM, st, maps, a,
                                          p.row_tiles, p.teams, by_group, shift, p.share);
    return e != cudaSuccess || !p.parts ? e : join_parts(type, a, p, by_group, st);
}

template <typename T, int DP>
cudaError_t rows_d(const AttendArgs &a, int type, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    const unsigned n = a.nodes * (a.q_heads / a.c.heads);
    if (n <= 16) return rows<T, DP, 1>(a, type, dev, st, bytes);
    // binary32 rows lie in two parts: with 64 of them one CTA fills an SM, and its four warps wait for one another's
    // products; with 32 there are two CTAs (136 rows of 96 entries: 930 us against 460)
    if constexpr (sizeof(T) == 2) {
        if (n > 32) return rows<T, DP, 4>(a, type, dev, st, bytes);
    }
    return rows<T, DP, 2>(a, type, dev, st, bytes);
}

template <typename T>
cudaError_t rows_t(const AttendArgs &a, int type, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    if (a.c.dim <= 64) return rows_d<T, 64>(a, type, dev, st, bytes);
    if (a.c.dim <= 128) return rows_d<T, 128>(a, type, dev, st, bytes);
    return rows_d<T, 256>(a, type, dev, st, bytes);
}

}  // namespace
}  // namespace attend
}  // namespace gbper
