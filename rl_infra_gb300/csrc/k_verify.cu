// k_verify.cu -- verification of drafted tokens.  One CTA takes one sequence: the accept tests, the
// total of the masses of the row it stops at (integers, so the order of summation does not
// matter), and the first place whose inclusive sum passes the mark.
#include "ops_internal.cuh"

namespace gbper {

namespace {

constexpr int kThreads = 256;
typedef unsigned long long u64;

// a mass in units of 2^-40: NaN and negative 0, above 1 as 1
__device__ __forceinline__ u64 units(float r)
{
    return r > 0.0f ? (u64)(fminf(r, 1.0f) * 1099511627776.0f) : 0ull;
}

template <typename T>
__device__ __forceinline__ u64 mass(const T *p, const T *q, long long without, unsigned j)
{
    const float v = to_f32(p[j]);
    if (q) return units(v - to_f32(q[j]));
    return (long long)j == without ? 0ull : units(v);
}

__device__ __forceinline__ u64 block_total(u64 v, u64 *red)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < kThreads / 32; ++w) v += red[w];
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_verify(VerifyArgs a)
{
    __shared__ u64 red[kThreads / 32], sums[kThreads];
    __shared__ int s_n, s_token;
    const long long b = blockIdx.x;
    const int t = threadIdx.x, D = a.drafts;
    const T *p = static_cast<const T *>(a.p) + b * a.sp[0];
    const T *q = a.q ? static_cast<const T *>(a.q) + b * a.sq[0] : nullptr;
    int m = a.lens ? a.lens[b] : D;
    m = max(0, min(m, D));
    if (t == 0) {
        s_n = m;
        s_token = -1;
    }
    __syncthreads();
    for (int i = t; i < D; i += kThreads) {
        const long long tok = load_index(a.tokens, b * a.stok + i, a.tok64);
        const bool in = tok >= 0 && tok < (long long)a.vocab;
        const float pt = in ? to_f32(p[i * a.sp[1] + tok]) : 0.0f;
        const float qt = !in ? 0.0f : q ? to_f32(q[i * a.sq[1] + tok]) : 1.0f;
        if (a.accept_p) a.accept_p[b * D + i] = i >= m || !in ? 0.0f : pt < qt ? pt / qt : 1.0f;
        if (i < m && !(in && __fmul_rn(a.u[b * a.su + i], qt) < pt)) atomicMin(&s_n, i);
    }
    __syncthreads();
    const int n = s_n;
    const T *pr = p + n * a.sp[1];
    const T *qr = nullptr;
    long long without = -1;
    if (n < m) {
        const long long tok = load_index(a.tokens, b * a.stok + n, a.tok64);
        if (tok < 0 || tok >= (long long)a.vocab) {
            if (t == 0 && a.status) atomicOr(a.status, PER_DEVFLAG_BAD_INDEX);
        } else {
            without = tok;
        }
        if (q) qr = q + n * a.sq[1];
    }
    const unsigned per = (a.vocab + kThreads - 1) / kThreads;
    const unsigned j0 = min(a.vocab, t * per), j1 = min(a.vocab, j0 + per);
    for (int pass = 0; pass < 2; ++pass) {
        u64 own = 0;
        for (unsigned j = j0; j < j1; ++j) own += mass(pr, qr, without, j);
        const u64 total = block_total(own, red);
        if (total == 0) {   // the target's own row
            qr = nullptr;
            without = -1;
            continue;
        }
        float u = a.us[b];
        const u64 U = u > 0.0f ? min((u64)(fminf(u, 1.0f) * 2147483648.0f), 0x7fffffffull) : 0ull;
        const u64 mark = U * (total >> 31) + ((U * (total & 0x7fffffffull)) >> 31);
        sums[t] = own;
        __syncthreads();
        u64 before = 0;
        for (int i = 0; i < t; ++i) before += sums[i];
        if (before <= mark && mark < before + own) {
            for (unsigned j = j0; j < j1; ++j) {
                before += mass(pr, qr, without, j);
                if (before > mark) {
                    s_token = (int)j;
                    break;
                }
            }
        }
        __syncthreads();
        break;
    }
    if (t == 0) a.accepted[b] = n;
    for (int i = t; i <= D; i += kThreads)
        a.out[b * (D + 1) + i] = i < n ? (int)load_index(a.tokens, b * a.stok + i, a.tok64) : i == n ? s_token : -1;
}

}  // namespace

cudaError_t launch_verify(int type, const VerifyArgs &a, cudaStream_t st)
{
    if (type == PER_TYPE_F32) k_verify<float><<<a.batch, kThreads, 0, st>>>(a);
    else if (type == PER_TYPE_F16) k_verify<__half><<<a.batch, kThreads, 0, st>>>(a);
    else k_verify<__nv_bfloat16><<<a.batch, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace gbper
