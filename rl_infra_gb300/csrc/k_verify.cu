// k_verify.cu -- verification of drafted tokens against the target's probabilities.
//
// Mathematics.  Token i passes when u_i q_i < p_i; the first that does not (or the end of the draft)
// fixes the row n, whose masses max(p - q, 0) (or p) are drawn from by their inclusive sum.  A mass
// counts in whole units of 2^-40: the sum of up to 2^18 of them fits in 64 bits and is the same in any
// order, so the draw can be split over CTAs and warps and still be one number, exactly.  The mark
// floor(U M / 2^31) with U < 2^31 is below M, and is taken in two 64-bit products.
//
// Work.  Two rows of V are all that has to be read (HBM bounds large batches; a chain of dependent loads
// bounds small ones: token, its probabilities, the rows, the place).  A sequence takes a cluster of
// 1 to 8 CTAs; each runs the accept tests for itself (a handful of loads, instead of a barrier), sums its
// part of the row, 16 bytes a load, and exchanges the sum through distributed shared memory (one
// hardware barrier).  The one warp whose stretch holds the mark reads its stretch again, from
// cache, and walks it with warp prefix sums.
//
// Measured (GB300): 512 sequences of 8 drafts over 131072 f32 102 us, 5.0 TB/s; one sequence of 4 over 32768 6.0 us.
#include "ops_internal.cuh"

#include <algorithm>

namespace gbper {

namespace {

typedef unsigned long long u64;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 4;   // 16-byte loads of each row that a lane has in flight

// Masses summed in units of 2^-40.  A mass r in [0, 1] is cut to hi 2^-20 + lo 2^-40 by two additions of
// 2^23 that round toward zero, whose low mantissa bits are the two whole numbers; the additions' bit
// patterns are summed as they are, and the pattern of 2^23 is taken off by the count.  (A conversion of a
// binary32 to 64 bits runs on the binary64 pipe, which bound the kernel: 56 us against 31 for 128
// sequences of 131072.)  Exact while a thread sums fewer than 2^12 masses: each adds at most 2^20 to a 32-bit sum.
static_assert(kMaxVocab / kThreads + 2 * 8 < 1u << 12, "a lane's masses: its share of a row and up to two pieces of 8");
struct Units {
    unsigned hi = 0, lo = 0;
    // r = max(0, min(1, p - q)); NaN counts 0
    __device__ __forceinline__ void add(float p, float q)
    {
        float r;
        asm("sub.rn.sat.f32 %0, %1, %2;" : "=f"(r) : "f"(p), "f"(q));
        const float a = __fmaf_rz(r, 1048576.0f, 8388608.0f);
        const float rest = fmaf(r, 1048576.0f, 8388608.0f - a);   // exact
        const float b = __fmaf_rz(rest, 1048576.0f, 8388608.0f);
        hi += __float_as_uint(a);
        lo += __float_as_uint(b);
    }
    __device__ __forceinline__ u64 total(unsigned n) const
    {
        return ((u64)(hi - n * 0x4b000000u) << 20) + (lo - n * 0x4b000000u);
    }
};

// 16 bytes at any address that is a multiple of 2: two aligned loads, shifted together.  The caller makes
// sure that both lie inside the row.  (Loads that memory keeps coherent: the read-only path is for what no kernel
// writes while this one runs, and this one begins before its predecessor in the stream has ended.)
__device__ __forceinline__ uint4 load_across(const unsigned char *p)
{
    const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u);
    const uint4 *a = reinterpret_cast<const uint4 *>(p - off);
    const uint4 lo = *a;
    if (off == 0) return lo;
    const uint4 hi = a[1];
    return shift_bytes(lo, hi, off);
}

// The row that is drawn from, in 16-byte pieces of p from the boundary at or before its start.
template <typename T>
struct Row {
    static constexpr int P = Pack<T>::N;
    const T *p, *q;         // q null: nothing is taken off
    long long without;      // a place that counts 0, or -1
    unsigned vocab, mis;

    // the values of p and q (0 without a q) of one piece; places outside the row give 0
    __device__ __forceinline__ void load(unsigned w, Pack<T> &a, Pack<T> &b) const
    {
        const long long j = (long long)w * P - mis;
        const bool inside = j >= 0 && j + P <= (long long)vocab;
        // the pieces around q's stretch must lie inside q's row too
        const bool margin = j >= P && j + 2 * P <= (long long)vocab;
        b.raw = make_uint4(0, 0, 0, 0);
        if (inside && (!q || margin)) {
            a.raw = *reinterpret_cast<const uint4 *>(p + j);
            if (q) b.raw = load_across(reinterpret_cast<const unsigned char *>(q + j));
        } else {
            float f[P], g[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const bool in = j + e >= 0 && j + e < (long long)vocab;
                f[e] = in ? to_f32(p[j + e]) : 0.0f;
                g[e] = in && q ? to_f32(q[j + e]) : 0.0f;
            }
            a.pack(f);   // exact: the values came from T
            b.pack(g);
        }
    }

    // p with the place that counts 0 taken out
    __device__ __forceinline__ void unpack(unsigned w, const Pack<T> &a, float *f) const
    {
        a.unpack(f);
        const long long k = without - ((long long)w * P - mis);
        if (without >= 0 && k >= 0 && k < P) {
#pragma unroll
            for (int e = 0; e < P; ++e)
                if (e == k) f[e] = 0.0f;
        }
    }

    __device__ __forceinline__ void add(unsigned w, const Pack<T> &a, const Pack<T> &b, Units &s) const
    {
        float f[P], g[P];
        unpack(w, a, f);
        b.unpack(g);
#pragma unroll
        for (int e = 0; e < P; ++e) s.add(f[e], g[e]);
    }
};

__device__ __forceinline__ u64 warp_sum(u64 v)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_verify(VerifyArgs a, unsigned csize, unsigned per_cta)
{
    constexpr int P = Pack<T>::N;
    __shared__ u64 warp_total[kWarps], cluster_total[2][kMaxCluster];
    __shared__ int s_n;
    const unsigned rank = blockIdx.x % csize;
    const long long b = blockIdx.x / csize;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, D = (int)a.drafts;
    if (t == 0) s_n = D;
    pdl_wait();
    pdl_release();
    if (csize > 1) cluster_arrive_relaxed();   // this CTA has started
    const T *p = static_cast<const T *>(a.p) + b * a.sp[0];
    const T *q = a.q ? static_cast<const T *>(a.q) + b * a.sq[0] : nullptr;
    const int m = a.lens ? max(0, min(a.lens[b], D)) : D;
    const float us = a.us[b];
    __syncthreads();
    for (int i = t; i < D; i += kThreads) {
        const long long tok = load_index(a.tokens, b * a.stok + i, a.tok64);
        const float u = a.u[b * a.su + i];
        const bool in = tok >= 0 && tok < (long long)a.vocab;
        const float pt = in ? to_f32(p[i * a.sp[1] + tok]) : 0.0f;
        const float qt = !in ? 0.0f : q ? to_f32(q[i * a.sq[1] + tok]) : 1.0f;
        if (a.accept_p && rank == 0) a.accept_p[b * D + i] = i >= m || !in ? 0.0f : pt < qt ? pt / qt : 1.0f;
        if (i < m && !(in && __fmul_rn(u, qt) < pt)) atomicMin(&s_n, i);
    }
    __syncthreads();
    const int n = min(s_n, m);

    Row<T> row;
    row.p = p + n * a.sp[1];
    row.q = nullptr;
    row.without = -1;
    row.vocab = a.vocab;
    row.mis = (unsigned)(reinterpret_cast<uintptr_t>(row.p) % 16 / sizeof(T));
    if (n < m) {
        const long long tok = load_index(a.tokens, b * a.stok + n, a.tok64);
        if (tok < 0 || tok >= (long long)a.vocab) {
            if (t == 0 && rank == 0 && a.status) atomicOr(a.status, PER_DEVFLAG_BAD_INDEX);
        } else if (!q) {
            row.without = tok;
        }
        if (q) row.q = q + n * a.sq[1];
    }
    if (rank == 0) {
        if (t == 0) a.accepted[b] = n;
        for (int i = t; i <= D; i += kThreads)
            if (i != n) a.out[b * (D + 1) + i] = i < n ? (int)load_index(a.tokens, b * a.stok + i, a.tok64) : -1;
    }

    const unsigned pieces = (row.mis + a.vocab + P - 1) / P;
    const unsigned v1 = min(pieces, (rank + 1) * per_cta);
    const unsigned per_warp = (per_cta + kWarps - 1) / kWarps;
    const unsigned w0 = min(rank * per_cta + warp * per_warp, v1), w1 = min(w0 + per_warp, v1);
    for (int attempt = 0; attempt < 2; ++attempt) {
        Units sum;
        unsigned count = 0;   // a lane's masses: at most 2^18 / (8 warps x 32 lanes), and a piece more
        for (unsigned w = w0 + lane; w < w1; w += 32 * kUnroll) {
            Pack<T> x[kUnroll], y[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                if (w + 32 * i < w1) row.load(w + 32 * i, x[i], y[i]);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                if (w + 32 * i < w1) {
                    row.add(w + 32 * i, x[i], y[i], sum);
                    count += P;
                }
        }
        const u64 own = warp_sum(sum.total(count));
        if (lane == 0) warp_total[warp] = own;
        __syncthreads();
        u64 mine = 0, before = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const u64 v = warp_total[i];
            mine += v;
            before += i < warp ? v : 0;
        }
        u64 total = mine;
        if (csize > 1) {
            if (attempt == 0) cluster_wait_acquire();   // every CTA of the sequence has started
            if (t < (int)csize) {
                const unsigned to = cluster_smem_addr(&cluster_total[attempt][rank], t);
                st_cluster_u32(to, (unsigned)mine);
                st_cluster_u32(to + 4, (unsigned)(mine >> 32));
            }
            cluster_sync_all();
            total = 0;
            for (unsigned r = 0; r < csize; ++r) {
                const u64 v = cluster_total[attempt][r];
                total += v;
                before += r < rank ? v : 0;
            }
        }
        if (total == 0) {
            if (attempt == 0 && (row.q || row.without >= 0)) {   // the target's own row
                row.q = nullptr;
                row.without = -1;
                __syncthreads();   // warp_total is read
                continue;
            }
            if (rank == 0 && t == 0) a.out[b * (D + 1) + n] = -1;
            return;
        }
        const u64 U = us > 0.0f ? min((u64)(fminf(us, 1.0f) * 2147483648.0f), 0x7fffffffull) : 0ull;
        const u64 mark = U * (total >> 31) + ((U * (total & 0x7fffffffull)) >> 31);
        if (mark < before || mark >= before + own) return;   // another warp's stretch
        for (unsigned w = w0; w < w1; w += 32 * kUnroll) {
            Pack<T> x[kUnroll], y[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                if (w + 32 * i + lane < w1) row.load(w + 32 * i + lane, x[i], y[i]);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const unsigned at = w + 32 * i + lane;
                Units piece;
                if (at < w1) row.add(at, x[i], y[i], piece);
                const u64 s = at < w1 ? piece.total(P) : 0;
                u64 incl = s;
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                if (mark < before + incl && mark >= before + incl - s) {
                    float f[P], g[P];
                    row.unpack(at, x[i], f);
                    y[i].unpack(g);
                    u64 c = before + incl - s;
                    int e = 0;
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        Units one;
                        one.add(f[k], g[k]);
                        c += one.total(1);
                        if (c <= mark) e = k + 1;
                    }
                    a.out[b * (D + 1) + n] = (int)((long long)at * P - row.mis + e);
                }
                before += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (mark < before) return;
        }
        return;
    }
}

template <typename T>
cudaError_t launch_t(const VerifyArgs &a, const DeviceInfo &dev, cudaStream_t st)
{
    constexpr unsigned P = 16 / sizeof(T);
    const unsigned pieces = (a.vocab + P - 1) / P + 1;   // a row that starts off a boundary has one more
    // CTAs for a sequence: more as long as each keeps at least 512 pieces (two a lane) and there are fewer than 8 an SM
    // in all (so fewer than 16 after the last doubling): each runs the accept tests again (512 sequences of 131072:
    // 4 CTAs a sequence 100 us, 8 103, 2 124)
    unsigned csize = 1;
    while (csize < kMaxCluster && pieces / csize > 1024 && (unsigned long long)a.batch * csize < 8ull * dev.sms) csize *= 2;
    return launch_clusters(k_verify<T>, a.batch * csize, kThreads, csize, 0, st, a, csize, (pieces + csize - 1) / csize);
}

}  // namespace

cudaError_t launch_verify(int type, const VerifyArgs &a, cudaStream_t st)
{
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    if (type == PER_TYPE_F32) return launch_t<float>(a, dev, st);
    if (type == PER_TYPE_F16) return launch_t<__half>(a, dev, st);
    return launch_t<__nv_bfloat16>(a, dev, st);
}

}  // namespace gbper
