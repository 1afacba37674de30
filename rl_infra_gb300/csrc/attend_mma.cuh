// attend_mma.cuh -- warp-wide matrix instructions of tree attention's kernels with few rows.
#pragma once

#include "attend.cuh"

#include <cstring>
#include <type_traits>

namespace gbper {
namespace attend {

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
// x = hi + lo: hi rounded to 11 bits, the rest rounded to 11 more (both cut where rounding would reach infinity or
// pass a NaN).  The instruction reads the upper 19 bits of each word.
__device__ __forceinline__ void split(float x, unsigned &hi, unsigned &lo)
{
    const unsigned b = __float_as_uint(x), half = (b & 0x7fffffffu) < 0x7f7ff000u ? 0x1000u : 0u;
    hi = (b + half) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) + half;
}

// Where piece c (16 bytes) of row r lies in a tile as the copy engine lays it: halves of 128 bytes of a head,
// [half][rows][128], each row's pieces turned by its number modulo 8.
__device__ __forceinline__ unsigned piece(unsigned rows, unsigned r, unsigned c)
{
    return (c >> 3) * rows * 128 + r * 128 + (((c & 7u) ^ (r & 7u)) << 4);
}

// piece c of a row of dim entries at src, entry by entry; zeros past the end and where there is no row
template <typename T>
__device__ __forceinline__ uint4 entries(const T *src, unsigned c, unsigned dim, bool some)
{
    constexpr int N = 16 / (int)sizeof(T);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (!some) return v;
    T e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = c * N + i < dim ? src[c * N + i] : from_f32<T>(0.0f);
    memcpy(&v, e, 16);
    return v;
}

// sc = q k for 16 rows from r0 of the m rows at qs, and KW keys from key0 of the kt at ks; `halves` of 128 bytes of a head
// (what lies past its entries is zero), four steps of the instruction each: without a branch between them, so that what
// one waits for does not keep the next.  binary32 queries lie in two parts, upper and lower.  A step of these takes two pieces four apart: column c of the instruction is entry 2 c
// mod 4 of piece c / 2 * 4, column c + 4 the entry behind it, so that 16 lanes read 16 different banks twice.
template <typename T, int DP, int KW>
__device__ __forceinline__ void scores(float (*sc)[4], const unsigned char *qs, unsigned m, unsigned r0, const unsigned char *ks,
                                       unsigned kt, unsigned key0, unsigned halves)
{
    const unsigned lane = threadIdx.x & 31u, g = lane >> 2, q4 = lane & 3u;
#pragma unroll
    for (int i = 0; i < KW / 8; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.0f;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            if (k % 4 == 0 && k / 4 >= (int)halves) break;
            unsigned qa[4];
            ldsm4(qa, smem_u32(qs + piece(m, r0 + (lane & 15u), k * 2 + (lane >> 4))));
#pragma unroll
            for (int i = 0; i < KW / 16; ++i) {
                unsigned kb[4];   // keys 0-7 and 8-15, entries 0-7 and 8-15 of each
                ldsm4(kb, smem_u32(ks + piece(kt, key0 + i * 16 + (lane & 7u) + ((lane >> 4) << 3), k * 2 + ((lane >> 3) & 1u))));
                mma16<T>(sc[2 * i], qa, kb[0], kb[1]);
                mma16<T>(sc[2 * i + 1], qa, kb[2], kb[3]);
            }
        }
    } else {
        // a sum for each kind of product and half of the steps, so that none waits for the one before it (and because the
        // instruction cuts its sums instead of rounding them: the shorter, the nearer)
        float low_q[KW / 8][4], low_k[KW / 8][4], odd[KW / 8][4];
#pragma unroll
        for (int i = 0; i < KW / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) low_q[i][e] = low_k[i][e] = odd[i][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < DP / 8; ++k) {
            if (k % 4 == 0 && k / 4 >= (int)halves) break;
            unsigned ah[4], al[4];
            const unsigned c = (k >> 2) * 8 + (k & 3) + (q4 >> 1) * 4, in = (q4 & 1u) * 8;
            const unsigned low = m * DP * 4;   // the lower parts lie behind the upper ones
            const uint2 x = *reinterpret_cast<const uint2 *>(qs + piece(m, r0 + g, c) + in);
            const uint2 y = *reinterpret_cast<const uint2 *>(qs + piece(m, r0 + g + 8, c) + in);
            const uint2 xl = *reinterpret_cast<const uint2 *>(qs + low + piece(m, r0 + g, c) + in);
            const uint2 yl = *reinterpret_cast<const uint2 *>(qs + low + piece(m, r0 + g + 8, c) + in);
            ah[0] = x.x, ah[1] = y.x, ah[2] = x.y, ah[3] = y.y;
            al[0] = xl.x, al[1] = yl.x, al[2] = xl.y, al[3] = yl.y;
#pragma unroll
            for (int i = 0; i < KW / 8; ++i) {
                const float2 z = *reinterpret_cast<const float2 *>(ks + piece(kt, key0 + i * 8 + g, c) + in);
                unsigned h0, l0, h1, l1;
                split(z.x, h0, l0);
                split(z.y, h1, l1);
                mma8(low_q[i], al, h0, h1);
                mma8(low_k[i], ah, l0, l1);
                mma8(k & 1 ? odd[i] : sc[i], ah, h0, h1);
            }
        }
#pragma unroll
        for (int i = 0; i < KW / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[i][e] = (sc[i][e] + odd[i][e]) + (low_q[i][e] + low_k[i][e]);
    }
}

// o += p v for the same rows and keys (p where the scores were).  TWO: 16-bit p in two parts, itself rounded and the rest rounded,
// so that what is lost of it is 2^-16 (float16 2^-22) and not a half step of the type.  Taken where it costs nothing, with one
// fragment of rows (64 sequences of up to 5000, one token, 153 us with it and without; one token over 1023 9.3 and 9.1); with
// two, the products no longer hide behind the copies (262145 tokens, 32 rows a head: 178 us and 171).  binary32: key 2 c is column c of the instruction,
// 2 c + 1 column c + 4: the scores lie so already.
template <typename T, int DP, int KW, bool TWO>
__device__ __forceinline__ void values(float (*o)[4], const float (*p)[4], const unsigned char *vs, unsigned kt, unsigned key0,
                                       unsigned halves)
{
    const unsigned lane = threadIdx.x & 31u, g = lane >> 2, q4 = lane & 3u;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < KW / 16; ++k) {
            const unsigned pa[4] = {pack2<T>(p[2 * k][0], p[2 * k][1]), pack2<T>(p[2 * k][2], p[2 * k][3]),
                                    pack2<T>(p[2 * k + 1][0], p[2 * k + 1][1]), pack2<T>(p[2 * k + 1][2], p[2 * k + 1][3])};
            unsigned pl[4];       // what is left of p
            if constexpr (TWO) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 hi = unpack2<T>(pa[j]);
                    pl[j] = pack2<T>(p[2 * k + (j >> 1)][(j & 1) * 2] - hi.x, p[2 * k + (j >> 1)][(j & 1) * 2 + 1] - hi.y);
                }
            }
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                if (i % 4 == 0 && i / 4 >= (int)halves) break;
                unsigned vb[4];   // keys 0-7 and 8-15 of entries 0-7, then of entries 8-15
                ldsm4t(vb, smem_u32(vs + piece(kt, key0 + k * 16 + (lane & 15u), i * 2 + (lane >> 4))));
                if constexpr (TWO) {
                    mma16<T>(o[2 * i], pl, vb[0], vb[1]);
                    mma16<T>(o[2 * i + 1], pl, vb[2], vb[3]);
                }
                mma16<T>(o[2 * i], pa, vb[0], vb[1]);
                mma16<T>(o[2 * i + 1], pa, vb[2], vb[3]);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < KW / 8; ++k) {
            unsigned ph[4], pl[4];
            split(p[k][0], ph[0], pl[0]);
            split(p[k][2], ph[1], pl[1]);
            split(p[k][1], ph[2], pl[2]);
            split(p[k][3], ph[3], pl[3]);
            constexpr int TOGETHER = 4;   // products whose sums are different ones, so that none waits for the one before it
#pragma unroll
            for (int i0 = 0; i0 < DP / 8; i0 += TOGETHER) {
                if (i0 / 4 >= (int)halves) break;
                unsigned h0[TOGETHER], l0[TOGETHER], h1[TOGETHER], l1[TOGETHER];
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j) {
                    const unsigned r = key0 + k * 8 + q4 * 2, c = (i0 + j) * 2 + (g >> 2), in = (g & 3u) * 4;
                    split(*reinterpret_cast<const float *>(vs + piece(kt, r, c) + in), h0[j], l0[j]);
                    split(*reinterpret_cast<const float *>(vs + piece(kt, r + 1, c) + in), h1[j], l1[j]);
                }
                float part[TOGETHER][4];      // eight keys' sum, added to the others' with rounding
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j) part[j][0] = part[j][1] = part[j][2] = part[j][3] = 0.0f;
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j) mma8(part[j], pl, h0[j], h1[j]);
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j) mma8(part[j], ph, l0[j], l1[j]);
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j) mma8(part[j], ph, h0[j], h1[j]);
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i0 + j][e] += part[j][e];
            }
        }
    }
}

// Hides the scores of a warp's keys that its rows' nodes (node < 0: no such row) do not see: first is the tile's first key,
// there(r) whether its key r has a page.  Every mask byte is asked for (places outside the tree clamped), so that none
// waits behind a branch for the one before it.
template <int KW, typename There>
__device__ __forceinline__ void hide(float (*sc)[4], const AttendArgs &a, unsigned b, const Span &s, const int *node, unsigned first,
                                     unsigned key0, There there)
{
    const unsigned q4 = threadIdx.x & 3u;
    const int nodes = s.total - s.len;                     // that the table has a place for
    const bool bytes = a.mask && nodes > 0;
    unsigned see[2] = {~0u, ~0u};                          // of the thread's columns, by node
    static_assert(KW / 4 <= 32, "");
    if (bytes) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint8_t *row = a.mask + b * a.sm[0] + (long long)max(node[e], 0) * a.sm[1];
            see[e] = 0;
#pragma unroll
            for (int i = 0; i < KW / 4; ++i) {
                const int j = (int)(first + key0 + (i >> 1) * 8 + q4 * 2 + (i & 1)) - s.len;
                see[e] |= row[min(max(j, 0), nodes - 1)] != 0 ? 1u << i : 0u;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned r = key0 + i * 8 + q4 * 2 + (e & 1);
            const int j = (int)(first + r) - s.len, n = node[e >> 1];
            const bool tree = bytes ? (see[e >> 1] >> (2 * i + (e & 1))) & 1u : j <= n;
            if (n < 0 || !(j < 0 || (j < nodes && tree)) || !there(r)) sc[i][e] = -INFINITY;
        }
}

// binary32 scores of keys that are seen and came out NaN, once more in plain sums: an infinite entry has no two parts (its rest
// is inf - inf), and its score may well be -inf.  row: of the rows that share a head of keys, the thread's first (rare: nothing
// here is fast).
template <int KW>
__device__ __forceinline__ void once_more(float (*sc)[4], const AttendArgs &a, unsigned b, unsigned h, unsigned group, const int *node,
                                          unsigned row, const unsigned char *ks, unsigned kt, unsigned key0)
{
    float all = 0.0f;
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) all += sc[i][e];
    if (!__any_sync(0xffffffffu, all != all)) return;
    const unsigned q4 = threadIdx.x & 3u;
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = node[e >> 1];
            if (sc[i][e] == sc[i][e] || n < 0) continue;
            const unsigned r = key0 + i * 8 + q4 * 2 + (e & 1), head = (h - (unsigned)n) * group + row + (e >> 1) * 8;
            const float *q = static_cast<const float *>(a.q) + b * a.sq[0] + n * a.sq[1] + head * a.sq[2];
            float s = 0.0f;
#pragma unroll 1
            for (unsigned d = 0; d < a.c.dim; ++d)
                s = fmaf(q[d], *reinterpret_cast<const float *>(ks + piece(kt, r, d >> 2) + (d & 3u) * 4), s);
            sc[i][e] = s * a.c2;
        }
}

// What a row's p and sum refer to, for its maximum so far (in log2).  p goes into a product as T: a float16 holds 11 bits down
// to 2^-14 and nothing below 2^-25, so that under one key far above the others theirs would be lost from the product, though
// not from the sum (8000 keys 18 nats below one whose value is 0: 0.5% off).  Referred to 2^-15 of the maximum, p uses the
// type's upper end too: 11 bits down to 2^-29 of the maximum, off by at most 2^-40 of it below.  (From 2^22 on the
// difference would be rounded.  bfloat16 and binary32 have the range: their p is at most 1.)
template <typename T>
__device__ __forceinline__ float below(float top)
{
    return std::is_same<T, __half>::value && fabsf(top) < 4194304.0f ? top - 15.0f : top;
}

// The softmax's step for a warp's scores sc (in log2 already), in place: maxima and sums of rows g and g + 8 carried on, o
// brought to the new maxima (p, sums and o refer to below(top)).  A thread's sums are its own columns' alone.
template <typename T, int DP, int KW>
__device__ __forceinline__ void soften(float (*sc)[4], float *top, float *sum, float (*o)[4])
{
    float keep[2], base[2], up[2] = {top[0], top[1]};
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) up[e >> 1] = fmaxf(up[e >> 1], sc[i][e]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        up[e] = fmaxf(up[e], __shfl_xor_sync(0xffffffffu, up[e], 1));
        up[e] = fmaxf(up[e], __shfl_xor_sync(0xffffffffu, up[e], 2));
        base[e] = up[e] == -INFINITY ? 0.0f : below<T>(up[e]);      // nothing seen yet: every p is 2^-inf = 0
        keep[e] = ex2(below<T>(top[e]) - base[e]);
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
    if (__any_sync(0xffffffffu, keep[0] != 1.0f || keep[1] != 1.0f)) {   // most tiles raise no maximum
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
            o[i][0] *= keep[0];
            o[i][1] *= keep[0];
            o[i][2] *= keep[1];
            o[i][3] *= keep[1];
        }
    }
}

// What was taken out of the values of key `key`, for the rows that see it (rare: nothing here is fast).
template <typename T, int DP>
__device__ __forceinline__ void give_back(const AttendArgs &a, unsigned b, const Span &s, const int *node, unsigned key, const T *v,
                                          float (*o)[4])
{
    const unsigned q4 = threadIdx.x & 3u;
    const bool see[2] = {node[0] >= 0 && sees(a, b, s, node[0], key), node[1] >= 0 && sees(a, b, s, node[1], key)};
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned d = i * 8 + q4 * 2 + (e & 1);
            if (d >= a.c.dim || !see[e >> 1]) continue;
            const float x = to_f32(v[d]);
            if (!finite(x)) o[i][e] += x;
        }
}

// Takes what is not finite (all bits of the exponent set) out of 16 bytes; whether there was any.
template <typename T>
__device__ __forceinline__ bool take_out(uint4 *at)
{
    constexpr unsigned E = sizeof(T) == 4 ? 0x7f800000u : std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    const uint4 v = *at;
    unsigned w[4] = {v.x, v.y, v.z, v.w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unsigned gone = 0;
        if (sizeof(T) == 4) {
            if ((w[i] & E) == E) gone = ~0u;
        } else {
            if ((w[i] & E & 0xffffu) == (E & 0xffffu)) gone |= 0xffffu;
            if ((w[i] & E & 0xffff0000u) == (E & 0xffff0000u)) gone |= 0xffff0000u;
        }
        any |= gone != 0;
        w[i] &= ~gone;
    }
    if (any) *at = make_uint4(w[0], w[1], w[2], w[3]);
    return any;
}

// The values of the sequence's end, in the tile at `vs` whose first key is `first`: zeros where there is no key, and what
// is not finite in a node's taken out.  Whether there was any.
template <typename T>
__device__ __forceinline__ bool clean(unsigned char *vs, unsigned kt, unsigned first, const Span &s, unsigned pieces, unsigned t, unsigned threads)
{
    const unsigned r0 = (unsigned)s.len > first ? (unsigned)s.len - first : 0;
    bool odd = false;
    for (unsigned u = t; u < (kt - r0) * pieces; u += threads) {
        const unsigned r = r0 + u / pieces, c = u % pieces;
        uint4 *at = reinterpret_cast<uint4 *>(vs + piece(kt, r, c));
        if (first + r >= (unsigned)s.total) *at = make_uint4(0, 0, 0, 0);
        else odd |= take_out<T>(at);
    }
    return odd;
}

}  // namespace attend
}  // namespace gbper
