// k_distill.cu -- the loss of a student's logits against a teacher's top logits, and its gradient.
//
// Mathematics.  With c = log2(e) / tau, a row's soft maximum is lse = m + tau ln s, m = max x, s =
// sum exp((x - m) / tau) = sum 2^((x - m) c); (m, s) of two stretches join by rescaling each s to the larger m, so one pass
// over a row suffices, split over threads, warps and CTAs, joined in a fixed order.  The differences
// are taken before they are scaled: x - m is exact where it matters and logits of the type's lowest
// value do not overflow.  -inf contributes 0; NaN and +inf make s NaN.
//   loss = tau sum_k q_k ((t_k - L) - (x_k - lse)),  grad_j = s_n tau (S p_j - q_j).
// Sums and normalisers are binary32; the gradient is rounded once.
//
// Work.  A row is split over a cluster of 1 to 8 CTAs.  Each CTA's loader warps copy their part of the
// row into shared memory (cp.async), keep the running (m, s) of what has arrived, exchange it with the row's
// other CTAs through distributed shared memory (one hardware barrier), and turn the part into the gradient
// on its way out.  So the step reads the logits once and writes the gradient once, which is its bound (HBM); three CTAs
// an SM are in different phases.  One more warp of each CTA handles the teacher's entries meanwhile; their q
// is taken off the gradient by a second write to those places after the CTA's barrier.  Every access to
// memory is 16 bytes on a 16-byte boundary but for a row's ends; a row that starts elsewhere (an odd
// vocabulary) keeps its place within the 16 bytes in shared memory and is shifted when it is read, so a row is
// summed in the same order, and gives the same bits, wherever it lies.  (Clusters that stay for many rows and
// load the next while they write this one were slower, 2.5 ms against 0.86 for 8192 rows of 131072: the
// barrier between the CTAs then waits for the stores of the row before.)
//
// Measured (GB300): step 8192 x 131072 bf16 with 64 entries 855 us, 5.0 TB/s, 74% of the copy rate; backward
// 2048 x 131072 bf16 87%, f32 89%; step of the latter 446 us, 71%; forward 32 x 1009 f32 3.4 us.
#include "ops_internal.cuh"

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

namespace gbper {

namespace {

constexpr int kMaxTop = 1024;
constexpr int kMaxCluster = 8;
// Loader warps of a CTA at most, CTAs an SM keeps registers for, and KB of a row that a CTA takes at most: 8, 3 and
// 64 take 0.86 ms for 8192 rows of 131072 bf16; 16 warps and 2 CTAs 1.17, 2 CTAs 1.10, 34 KB (more and smaller CTAs
// in larger clusters) 1.34.
constexpr int kMaxWarps = 8, kCtasPerSm = 3, kPartKb = 64;
constexpr int kUnroll = 4;       // pieces of 16 bytes a loader thread takes at a time
constexpr int kAhead = 1;        // batches of them under way at a time, the one that is waited for among them (0.86 ms; 4: 0.90)
constexpr float kInf = __builtin_huge_valf();
// A normaliser at or below this is of a row that a mask leaves nothing of: all its logits are -inf, or about the lowest value
// of binary32 or bfloat16, where m + tau ln s is m and no p can be told from it.
constexpr float kNothing = -0x1p100f;

struct RowSum {
    float m, s;
};

// log2(e) / tau in two parts: the nearest binary32 and what that leaves
struct Scale {
    float c, rest;
};

__device__ __forceinline__ float finite_or_zero(float m) { return m == -kInf ? 0.0f : m; }

// exp(d / tau) of two differences (-inf gives 0, NaN stays).  The power of 2 is good to 2^-22; the rounding of its
// argument takes a relative |d / tau| 2^-24 more (4e-6 at 60), which MORE makes up for by the first order of what
// it left out.  The gradient of binary32 elements and the teacher's q have that.  Sums do not: with p the share of
// a term, sum p |d / tau| = H(p) - ln s <= ln V, so a sum is off by at most ln V 2^-24 for it (and with it, forward
// 2048 x 131072 f32 took 315 us against 267).  Nor have 16-bit gradients, rounded to 2^-9 or 2^-12 in the end.
template <bool MORE>
__device__ __forceinline__ F2 exps(F2 d, Scale k)
{
    const F2 minus_x = d * F2{-k.c, -k.c};
    F2 v{ex2(-minus_x.x), ex2(-minus_x.y)};
    if constexpr (MORE) {
        constexpr float kLn2 = 0.693147182f;
        F2 r = fma2(d, F2{k.rest, k.rest}, fma2(d, F2{k.c, k.c}, minus_x)) * F2{kLn2, kLn2};
        // (infinite or NaN where x is -inf: the power is 0 then, and stays; a NaN in d is in v)
        r.x = fminf(r.x, 1.0f);
        r.y = fminf(r.y, 1.0f);
        v = fma2(v, r, v);
    }
    return v;
}

template <bool MORE>
__device__ __forceinline__ float exps(float d, Scale k)
{
    return exps<MORE>(F2{d, 0.0f}, k).x;
}

__device__ __forceinline__ RowSum join(RowSum a, RowSum b, Scale c)
{
    RowSum r;
    r.m = fmaxf(a.m, b.m);
    const float e = finite_or_zero(r.m);
    r.s = a.s * exps<false>(a.m - e, c) + b.s * exps<false>(b.m - e, c);
    return r;
}

__device__ __forceinline__ void copy16(void *smem, const void *global)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(smem)), "l"(global) : "memory");
}

// what contributes nothing
template <typename T>
__device__ __forceinline__ Pack<T> nothing()
{
    float f[Pack<T>::N];
#pragma unroll
    for (int e = 0; e < Pack<T>::N; ++e) f[e] = -kInf;
    Pack<T> r;
    r.pack(f);
    return r;
}

// the elements from j on that lie before `end`, element by element
template <typename T>
__device__ __forceinline__ Pack<T> ragged_end(const T *x, int j, int end)
{
    float f[Pack<T>::N];
#pragma unroll
    for (int e = 0; e < Pack<T>::N; ++e) f[e] = j + e < end ? to_f32(x[j + e]) : -kInf;
    Pack<T> r;
    r.pack(f);   // exact: the values came from T
    return r;
}

// A thread's running maximum and sums of two lanes of pairs, rescaled where the maximum rises.
template <typename T>
struct Running {
    static constexpr int P = Pack<T>::N;
    float m = -kInf;
    F2 s0 = {0.0f, 0.0f}, s1 = {0.0f, 0.0f};

    // the largest of a batch (NaN never raises it: it stays in the sums)
    static __device__ __forceinline__ float largest(const Pack<T> (&in)[kUnroll])
    {
        if constexpr (sizeof(T) == 2) {   // pairs, in their own type
            typedef typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type Two;
            Two r;
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const unsigned w[4] = {in[i].raw.x, in[i].raw.y, in[i].raw.z, in[i].raw.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    Two v;
                    memcpy(&v, &w[k], 4);
                    r = i + k ? __hmax2(r, v) : v;
                }
            }
            const float a = to_f32(r.x), b = to_f32(r.y);
            return fmaxf(fmaxf(a, b), -kInf);   // (both NaN)
        } else {
            float r = -kInf;
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                float f[P];
                in[i].unpack(f);
#pragma unroll
                for (int e = 0; e < P; ++e) r = fmaxf(r, f[e]);
            }
            return r;
        }
    }
    __device__ __forceinline__ void add(const Pack<T> (&in)[kUnroll], Scale c)
    {
        const float b = largest(in);
        if (b > m) {
            const float k = exps<false>(m - b, c);   // 0 at first
            s0 = s0 * F2{k, k};
            s1 = s1 * F2{k, k};
            m = b;
        }
        const float r = -finite_or_zero(m);
        const F2 ref{r, r};
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            float f[P];
            in[i].unpack(f);
#pragma unroll
            for (int e = 0; e < P; e += 2) {
                const F2 v = exps<false>(F2{f[e], f[e + 1]} + ref, c);
                if (e & 2) s1 = s1 + v;
                else s0 = s0 + v;
            }
        }
    }
    __device__ __forceinline__ RowSum sum() const
    {
        const F2 s = s0 + s1;
        return {m, s.x + s.y};
    }
};

// P consecutive elements of a part in shared memory from element j on (j + P is the next lane's j; the whole
// warp calls), of which those in [lo, hi) are there; the others give -inf.  p + j need not be on a 16-byte
// boundary: the blocks on boundaries are read, and joined with the next lane's.
template <typename T>
struct Pieces {
    static constexpr int P = Pack<T>::N;
    const T *p;
    int lo, hi;
    unsigned off;   // bytes from the boundary at or before p + j
    uint4 a[kUnroll], b[kUnroll];

    __device__ __forceinline__ Pieces(const T *p_, int lo_, int hi_, int j)
        : p(p_), lo(lo_), hi(hi_), off((unsigned)(reinterpret_cast<uintptr_t>(p_ + j) & 15u))
    {
    }
    static __device__ __forceinline__ uint4 load(const void *p) { return *static_cast<const uint4 *>(p); }
    __device__ __forceinline__ int before() const { return (int)(off / (unsigned)sizeof(T)); }
    __device__ __forceinline__ bool whole(int j) const { return j >= lo && j + P <= hi; }
    // every block that the pieces from element `first` to element `last` need may be read
    __device__ __forceinline__ bool whole_blocks(int first, int last) const
    {
        return first - before() >= lo && last - before() + (off ? 2 * P : P) <= hi;
    }
    __device__ __forceinline__ void request(int i, int j)
    {
        const int first = j - before();
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        if (whole(first)) a[i] = load(p + first);
        if (off && (threadIdx.x & 31) == 31 && whole(first + P)) b[i] = load(p + first + P);
    }
    // pieces w, w + step, ... of P elements counted from p (whole_blocks)
    __device__ __forceinline__ void request_all(int w, int step, int shift = 0)
    {
        const unsigned char *from = reinterpret_cast<const unsigned char *>(p + shift) - off + (long long)w * 16;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) a[i] = load(from + i * step * 16);
        if (off && (threadIdx.x & 31) == 31) {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) b[i] = load(from + i * step * 16 + 16);
        }
    }
    // the whole warp calls
    __device__ __forceinline__ Pack<T> shifted(int i) const
    {
        Pack<T> r;
        r.raw = a[i];
        if (off) {
            const uint4 n = make_uint4(__shfl_down_sync(0xffffffffu, a[i].x, 1), __shfl_down_sync(0xffffffffu, a[i].y, 1),
                                       __shfl_down_sync(0xffffffffu, a[i].z, 1), __shfl_down_sync(0xffffffffu, a[i].w, 1));
            r.raw = shift_bytes(a[i], (threadIdx.x & 31) == 31 ? b[i] : n, off);
        }
        return r;
    }
    __device__ __forceinline__ Pack<T> get(int i, int j) const
    {
        const Pack<T> r = shifted(i);
        const int first = j - before();
        return whole(first) && (!off || whole(first + P)) ? r : ragged(j);
    }
    // element by element
    __device__ __forceinline__ Pack<T> ragged(int j) const
    {
        float f[P];
#pragma unroll
        for (int e = 0; e < P; ++e) f[e] = j + e >= lo && j + e < hi ? to_f32(p[j + e]) : -kInf;
        Pack<T> r;
        r.pack(f);   // exact: the values came from T
        return r;
    }
};

// The join of n stretches: the largest maximum first, then the rescaled sums in their order.
__device__ __forceinline__ RowSum gather(const RowSum *p, int n, Scale c)
{
    RowSum r{-kInf, 0.0f};
    for (int i = 0; i < n; ++i) r.m = fmaxf(r.m, p[i].m);
    const float e = finite_or_zero(r.m);
    for (int i = 0; i < n; ++i) r.s += p[i].s * exps<false>(p[i].m - e, c);
    return r;
}

// Static shared memory of a CTA (the dynamic part: the CTA's part of the row, then the teacher's entries).
struct Shared {
    RowSum cluster[kMaxCluster];
    RowSum warp[kMaxWarps];
    float S;
    int some, repeated;
};

__device__ __forceinline__ unsigned hash_place(int at, unsigned mask) { return ((unsigned)at * 2654435761u >> 12) & mask; }

template <typename T, int PART>
__global__ void __launch_bounds__((kMaxWarps + 1) * 32, kCtasPerSm) k_distill(DistillArgs a, unsigned csize, unsigned per_cta,
                                                                  unsigned hash_size)
{
    constexpr int P = Pack<T>::N;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ Shared sh;
    uint4 *part = reinterpret_cast<uint4 *>(dyn);                             // [per_cta + 1]
    float *q = reinterpret_cast<float *>(dyn + ((size_t)per_cta + 1) * 16);   // [K]
    float *d = q + a.k;                                                       // [K] t - L
    float *xk = d + a.k;                                                      // [K] the student's logits there
    int *at = reinterpret_cast<int *>(xk + a.k);                              // [K] place, -1: left out
    int *table = at + a.k;                                                    // [hash_size]
    const int K = (int)a.k;
    const unsigned rank = blockIdx.x % csize;   // also the CTA's rank in its cluster, where there is one
    const long long row = blockIdx.x / csize;
    const Scale c{a.c, a.c_rest};
    const int loaders = (int)blockDim.x - 32, t = (int)threadIdx.x, lane = t & 31;
    pdl_wait();
    pdl_release();
    if (csize > 1 && PART != kDistillBackward) cluster_arrive_relaxed();   // this CTA has started

    const T *x = static_cast<const T *>(a.x) + row * a.sx;
    // the row in pieces of P elements; this CTA takes pieces [v0, v1), which are elements [j0, j1)
    const unsigned pieces = (a.vocab + P - 1) / P;
    const unsigned v0 = min(rank * per_cta, pieces), v1 = min(v0 + per_cta, pieces);
    const int j0 = (int)(v0 * P), j1 = (int)min(v1 * P, a.vocab);

    // element j of the part is cells[j]
    const int mis = (int)(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
    const T *cells = reinterpret_cast<const T *>(part) + mis - j0;

    RowSum own{-kInf, 0.0f};
    if (t >= loaders) {
        // ---- the teacher's entries -----------------------------------------------------------
        if (PART != kDistillForward)
            for (unsigned i = lane; i < hash_size; i += 32) table[i] = -1;
        float tm = -kInf;
        for (int k = lane; k < K; k += 32) {
            long long i = load_index(a.idx, row * a.si + k, a.idx64);
            float v = load_typed(a.top, row * a.st + k, a.top_type);
            if (i >= (long long)a.vocab) {
                if (a.status && rank == 0) atomicOr(a.status, PER_DEVFLAG_BAD_INDEX);
                i = -1;
            }
            if (i < 0) {
                i = -1;
                v = -kInf;
            }
            at[k] = (int)i;
            d[k] = v;
            // (the loss needs every entry's logit, the gradient those of the CTA's own part, which it holds)
            if (PART != kDistillBackward && rank == 0) xk[k] = i >= 0 ? to_f32(x[i]) : 0.0f;
            tm = fmaxf(tm, v);
        }
        for (int o = 16; o; o >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
        // log q = (t - e) - l: the difference from the largest first, so that what all entries share costs no digits
        float e, l;
        if (a.teacher_lse) {
            e = a.teacher_lse[row];
            l = 0.0f;
        } else {
            e = finite_or_zero(tm);
            float s = 0.0f;
            for (int k = lane; k < K; k += 32) s += exps<true>(d[k] - e, c);
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            l = s == 0.0f ? 0.0f : a.tau * logf(s);
        }
        float S = 0.0f;
        for (int k = lane; k < K; k += 32) {
            const float v = (d[k] - e) - l, w = at[k] >= 0 ? exps<true>(v, c) : 0.0f;
            d[k] = v;
            q[k] = w;
            S += w;
        }
        for (int o = 16; o; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
        int repeated = 0;
        if (PART != kDistillForward) {
            // does a place stand twice among the entries?  open addressing, at most half full
            __syncwarp();
            for (int k = lane; k < K; k += 32) {
                const int p = at[k];
                if (p < 0) continue;
                for (unsigned h = hash_place(p, hash_size - 1);; h = (h + 1) & (hash_size - 1)) {
                    const int was = atomicCAS(&table[h], -1, p);
                    if (was == p) repeated = 1;
                    if (was == -1 || was == p) break;
                }
            }
            repeated = __any_sync(0xffffffffu, repeated);
        }
        if (lane == 0) {
            sh.S = S;
            sh.some = !(S == 0.0f);
            sh.repeated = repeated;
        }
    } else {
        // ---- this CTA's part of the row: pieces v + i loaders + lane of each batch ------------------
        Running<T> run;
        const unsigned base = v0 + (t & ~31), step = loaders * kUnroll;
        const unsigned inner = (kUnroll - 1) * loaders + 32;   // pieces from a warp's first to its last of a batch
        if (mis == 0) {
            auto request = [&](unsigned v) {
                if ((int)((v + inner) * P) <= j1) {
                    uint4 *to = part + (v + lane - v0);
                    const T *src = x + (size_t)(v + lane) * P;
#pragma unroll
                    for (int i = 0; i < kUnroll; ++i) copy16(to + i * loaders, src + (size_t)(i * loaders) * P);
                } else {
#pragma unroll 1
                    for (int i = 0; i < kUnroll; ++i) {
                        const unsigned w = v + i * loaders + lane;
                        if ((int)((w + 1) * P) <= j1) copy16(&part[w - v0], x + (size_t)w * P);
                        else if (w < v1) part[w - v0] = ragged_end(x, (int)(w * P), j1).raw;
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
#pragma unroll
            for (int b = 0; b < kAhead; ++b) request(base + b * step);
            for (unsigned v = base; v < v1; v += step) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
                if (PART != kDistillBackward) {
                    Pack<T> in[kUnroll];
                    if (v + inner <= v1) {
                        const uint4 *at = part + (v + lane - v0);
#pragma unroll
                        for (int i = 0; i < kUnroll; ++i) in[i].raw = at[i * loaders];
                        run.add(in, c);
                    } else {
#pragma unroll
                        for (int i = 0; i < kUnroll; ++i) {
                            const unsigned w = v + i * loaders + lane;
                            in[i] = nothing<T>();
                            if (w < v1) in[i].raw = part[w - v0];
                        }
                        run.add(in, c);
                    }
                }
                request(v + kAhead * step);
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        } else {
            // off a boundary: the blocks on boundaries that hold the part, each element as far from one as in
            // memory; block w holds elements j0 - mis + w P and on.  Any thread's piece lies in two blocks, so
            // all of them come first.
            const T *src = x + (j0 - mis);
            const int blocks = j0 < j1 ? (j1 - j0 + mis + P - 1) / P : 0;
            const int lo = j0 == 0 ? 1 : 0, whole = min(blocks, ((int)a.vocab - j0 + mis) / P);   // the row's own
            for (int w = t; w < blocks; w += loaders) {
                if (w >= lo && w < whole) {
                    copy16(&part[w], src + (size_t)w * P);
                } else {
                    T *to = reinterpret_cast<T *>(&part[w]);
#pragma unroll 1
                    for (int e = 0; e < P; ++e) {
                        const int j = j0 - mis + w * P + e;
                        if (j >= j0 && j < j1) to[e] = x[j];
                    }
                }
            }
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;\n\tbar.sync 1, %0;" ::"r"(loaders) : "memory");
            if (PART != kDistillBackward) {
                Pieces<T> held(cells, j0, j1, j0);
                for (unsigned v = base; v < v1; v += step) {
                    Pack<T> in[kUnroll];
                    if ((int)((v + inner) * P) <= j1 && held.whole_blocks((int)(v * P), (int)((v + inner - 1) * P))) {
                        held.request_all((int)v + lane, loaders);
#pragma unroll
                        for (int i = 0; i < kUnroll; ++i) in[i] = held.shifted(i);
                    } else {
#pragma unroll
                        for (int i = 0; i < kUnroll; ++i) held.request(i, (int)((v + i * loaders + lane) * P));
#pragma unroll
                        for (int i = 0; i < kUnroll; ++i) in[i] = held.get(i, (int)((v + i * loaders + lane) * P));
                    }
                    run.add(in, c);
                }
            }
        }
        if (PART != kDistillBackward) {
            own = run.sum();
            for (int o = 16; o; o >>= 1) {
                RowSum other{__shfl_xor_sync(0xffffffffu, own.m, o), __shfl_xor_sync(0xffffffffu, own.s, o)};
                // the lower lane's stretch first, so that both lanes get the same bits
                own = (lane & o) ? join(other, own, c) : join(own, other, c);
            }
            if (lane == 0) sh.warp[t >> 5] = own;
        }
    }
    __syncthreads();
    float lse;
    RowSum all{-kInf, 0.0f};
    if (PART != kDistillBackward) {
        const int warps = loaders / 32;
        if (csize == 1) {
            all = gather(sh.warp, warps, c);
        } else {
            cluster_wait_acquire();   // every CTA of the row has started
            if (t < (int)csize) {
                all = gather(sh.warp, warps, c);
                const unsigned to = cluster_smem_addr(&sh.cluster[rank], t);
                st_cluster_f32(to, all.m);
                st_cluster_f32(to + 4, all.s);
            }
            cluster_sync_all();
            all = gather(sh.cluster, (int)csize, c);
        }
        const float m = finite_or_zero(all.m), l = a.tau * logf(all.s);
        lse = all.s == 0.0f ? -kInf : m + l;
        if (rank == 0 && t >= loaders) {
            float loss = 0.0f;
            for (int k = lane; k < K; k += 32)
                if (q[k] != 0.0f) loss += q[k] * a.tau * (d[k] - ((xk[k] - m) - l));   // (tau first: it may keep it finite)
            for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
            if (lane == 0) {
                a.loss[row] = sh.some && !(lse <= kNothing) ? loss : 0.0f;
                if (a.lse) a.lse[row] = lse;
            }
        }
    } else {
        lse = a.lse[row];
    }
    if (PART == kDistillForward) return;

    // ---- the gradient of this CTA's part --------------------------------------------------------
    const bool live = sh.some && !(lse <= kNothing);   // (NaN is)
    const float g = (a.scale ? a.scale[row] : 1.0f) * a.tau;
    // from lse in the step too: it gives the same bits as the forward and the backward call
    const float f0 = live ? g * sh.S : 0.0f;
    T *out = static_cast<T *>(a.grad) + row * a.sg;
    // pieces of the output's own 16-byte boundaries; those that another CTA or row shares are written
    // element by element
    const int misg = (int)(reinterpret_cast<uintptr_t>(out) % 16 / sizeof(T));
    if (t < loaders && j0 < j1) {
        const int o0 = (j0 + misg) / P, o1 = (j1 - 1 + misg) / P + 1, first = o0 + (t & ~31), step = loaders * kUnroll;
        const F2 ref{-lse, -lse}, ff{f0, f0};
        Pieces<T> from(cells, j0, j1, o0 * P - misg);
        auto turn = [&](Pack<T> &in) {
            float f[P];
            in.unpack(f);
#pragma unroll
            for (int e = 0; e < P; e += 2) {
                const F2 y = exps<sizeof(T) == 4>(F2{f[e], f[e + 1]} + ref, c) * ff;
                f[e] = y.x;
                f[e + 1] = y.y;
            }
            in.pack(f);
        };
        auto ragged = [&](int j, Pack<T> in) {   // the ends of the part
            float f[P];
            in.unpack(f);
#pragma unroll
            for (int e = 0; e < P; ++e)
                if (j + e >= j0 && j + e < j1) out[j + e] = from_f32<T>(f[e]);   // exact
        };
        if (!live) {
            for (int v = first; v < o1; v += loaders) {
                const int j = (v + lane) * P - misg;
                Pack<T> zero;
                zero.raw = make_uint4(0, 0, 0, 0);
                if (j >= j0 && j + P <= j1) *reinterpret_cast<uint4 *>(out + j) = zero.raw;
                else ragged(j, zero);
            }
        } else {
            for (int v = first; v < o1; v += step) {
                Pack<T> in[kUnroll];
                const int last = v + (kUnroll - 1) * loaders + 31;
                if (v * P - misg >= j0 && (last + 1) * P - misg <= j1 && from.whole_blocks(v * P - misg, last * P - misg)) {
                    uint4 *to = reinterpret_cast<uint4 *>(out - misg) + v + lane;
                    if (from.off == 0) {
                        const uint4 *at = reinterpret_cast<const uint4 *>(cells - misg) + v + lane;
#pragma unroll
                        for (int i = 0; i < kUnroll; ++i) in[i].raw = at[i * loaders];
                    } else {
                        from.request_all(v + lane, loaders, -misg);
#pragma unroll
                        for (int i = 0; i < kUnroll; ++i) in[i] = from.shifted(i);
                    }
#pragma unroll
                    for (int i = 0; i < kUnroll; ++i) {
                        turn(in[i]);
                        to[i * loaders] = in[i].raw;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kUnroll; ++i) from.request(i, (v + i * loaders + lane) * P - misg);
#pragma unroll
                    for (int i = 0; i < kUnroll; ++i) {
                        const int j = (v + i * loaders + lane) * P - misg;
                        in[i] = from.get(i, j);
                        turn(in[i]);
                        if (j >= j0 && j + P <= j1) *reinterpret_cast<uint4 *>(out + j) = in[i].raw;
                        else ragged(j, in[i]);
                    }
                }
            }
        }
    }
    if (!live) return;
    __syncthreads();   // the places of the entries below are written
    for (int k = t; k < K; k += (int)blockDim.x) {
        const int p = at[k];
        if (p < j0 || p >= j1) continue;   // left out, or another CTA's
        float sum = q[k];
        if (sh.repeated) {   // entries that name one place: the first of them takes all, in their order
            bool first = true;
            sum = 0.0f;
            for (int i = 0; i < K; ++i)
                if (at[i] == p) {
                    first = first && i >= k;
                    sum += q[i];
                }
            if (!first) continue;
        }
        const float v = to_f32(cells[p]);
        out[p] = from_f32<T>(f0 * exps<sizeof(T) == 4>(v - lse, c) - g * sum);
    }
}

// The largest dynamic shared memory a launch may ask for, set once per device.
constexpr size_t kMaxPart = 160 * 1024;
constexpr size_t kMaxDyn = kMaxPart + kMaxTop * 16 + 2 * kMaxTop * 4;

template <typename T>
cudaError_t attributes()
{
    cudaError_t e = cudaFuncSetAttribute(k_distill<T, kDistillForward>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxDyn);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_distill<T, kDistillBackward>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxDyn);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_distill<T, kDistillStep>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxDyn);
    return e;
}

cudaError_t init_once(int device)
{
    static std::atomic<bool> done[64];   // (two threads may both set the attributes, to the same values)
    if (done[device].load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = attributes<float>();
    if (e == cudaSuccess) e = attributes<__half>();
    if (e == cudaSuccess) e = attributes<__nv_bfloat16>();
    if (e == cudaSuccess) done[device].store(true, std::memory_order_release);
    return e;
}

template <typename T>
cudaError_t launch_t(DistillPart part, const DistillArgs &a, const DeviceInfo &dev, cudaStream_t st)
{
    constexpr unsigned P = 16 / sizeof(T);
    const unsigned pieces = (a.vocab + P - 1) / P;
    // CTAs for a row: enough that its part takes at most 64 KB of shared memory (three CTAs an SM, so
    // that one writes while others read), and that few rows still fill the SMs
    unsigned csize = 1;
    while (csize < kMaxCluster && (pieces + csize - 1) / csize * 16 > kPartKb * 1024) csize *= 2;
    while (csize < kMaxCluster && a.rows * csize < 2ull * dev.sms && pieces / csize > 512) csize *= 2;
    const unsigned per_cta = (pieces + csize - 1) / csize;
    if (a.rows * csize > 0x7fffffffull) return cudaErrorInvalidConfiguration;
    unsigned warps = 1;
    while (warps < (unsigned)kMaxWarps && warps * 32 * kUnroll < per_cta) warps *= 2;
    unsigned hash_size = 0;
    if (part != kDistillForward) {
        hash_size = 32;
        while (hash_size < 2 * a.k) hash_size *= 2;
    }
    const size_t smem = ((size_t)per_cta + 1) * 16 + (size_t)a.k * 16 + (size_t)hash_size * 4;
    const unsigned grid = (unsigned)(a.rows * csize), block = (warps + 1) * 32;
    if (part == kDistillForward)
        return launch_clusters(k_distill<T, kDistillForward>, grid, block, csize, smem, st, a, csize, per_cta, hash_size);
    if (part == kDistillBackward)
        return launch_clusters(k_distill<T, kDistillBackward>, grid, block, 1, smem, st, a, csize, per_cta, hash_size);
    return launch_clusters(k_distill<T, kDistillStep>, grid, block, csize, smem, st, a, csize, per_cta, hash_size);
}

}  // namespace

cudaError_t launch_distill(int type, DistillPart part, const DistillArgs &a, cudaStream_t st)
{
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    if (e == cudaSuccess) e = init_once(dev.device);
    if (e != cudaSuccess) return e;
    if (type == PER_TYPE_F32) return launch_t<float>(part, a, dev, st);
    if (type == PER_TYPE_F16) return launch_t<__half>(part, a, dev, st);
    return launch_t<__nv_bfloat16>(part, a, dev, st);
}

}  // namespace gbper
