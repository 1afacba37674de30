// k_distill.cu -- the loss of a student's logits against a teacher's top logits, and its gradient.
// One CTA takes one row: the teacher's entries are normalised in shared memory, the row's soft
// maximum is one pass with a running maximum and sum, the gradient a second pass.
#include "ops_internal.cuh"

namespace gbper {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTop = 1024;
constexpr float kInf = __builtin_huge_valf();

// (m, s) of two stretches: the maximum and the sum of 2^((x - maximum) c)
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2, float c)
{
    const float mm = fmaxf(m, m2);
    if (mm == -kInf) return;   // both empty (NaN never raises a maximum: it stays in the sum)
    s = (m == -kInf ? s : s * exp2f((m - mm) * c)) + (m2 == -kInf ? s2 : s2 * exp2f((m2 - mm) * c));
    m = mm;
}

__device__ __forceinline__ float block_sum(float v, float *red)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kThreads / 32; ++w) v += red[w];
    return v;
}

__device__ __forceinline__ float block_max(float v, float *red)
{
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kThreads / 32; ++w) v = fmaxf(v, red[w]);
    return v;
}

template <typename T, int PART>
__global__ void __launch_bounds__(kThreads) k_distill(DistillArgs a)
{
    __shared__ float q[kMaxTop], d[kMaxTop], xk[kMaxTop];
    __shared__ int at[kMaxTop];
    __shared__ float red[2 * (kThreads / 32)];
    const long long row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.sx;
    const int t = threadIdx.x, K = a.k;
    const float c = kLog2e / a.tau;
    // the teacher's row: q, log q as a difference, the student's logits at its places
    float tm = -kInf;
    for (int k = t; k < K; k += kThreads) {
        long long i = load_index(a.idx, row * a.si + k, a.idx64);
        if (i >= (long long)a.vocab) {
            if (a.status) atomicOr(a.status, PER_DEVFLAG_BAD_INDEX);
            i = -1;
        }
        if (i < 0) i = -1;
        at[k] = (int)i;
        d[k] = i < 0 ? -kInf : load_typed(a.top, row * a.st + k, a.top_type);
        xk[k] = i < 0 ? 0.0f : to_f32(x[i]);
        tm = fmaxf(tm, d[k]);
    }
    tm = block_max(tm, red);
    float L;
    if (a.teacher_lse) {
        L = a.teacher_lse[row];
    } else {
        float s = 0.0f;
        for (int k = t; k < K; k += kThreads)
            if (at[k] >= 0 && tm != -kInf) s += exp2f((d[k] - tm) * c);
            else if (at[k] >= 0) s += d[k] == d[k] ? 0.0f : d[k];
        s = block_sum(s, red);
        L = tm + a.tau * logf(s);
        if (tm == -kInf) L = s == s ? 0.0f : s;
    }
    float S = 0.0f;
    for (int k = t; k < K; k += kThreads) {
        d[k] -= L;
        q[k] = at[k] >= 0 ? exp2f(d[k] * c) : 0.0f;
        S += q[k];
    }
    S = block_sum(S, red);
    const bool some = !(S == 0.0f);
    float m = -kInf, s = 0.0f;
    float lse;
    if (PART != kDistillBackward) {
        for (unsigned j = t; j < a.vocab; j += kThreads) {
            const float v = to_f32(x[j]);
            if (v > m) {
                s *= exp2f((m - v) * c);
                m = v;
            }
            if (m != -kInf) s += exp2f((v - m) * c);
            else if (!(v == v)) s = v;
        }
        for (int o = 16; o; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
            join(m, s, m2, s2, c);
        }
        __syncthreads();
        if ((t & 31) == 0) {
            red[2 * (t >> 5)] = m;
            red[2 * (t >> 5) + 1] = s;
        }
        __syncthreads();
        m = red[0];
        s = red[1];
        for (int w = 1; w < kThreads / 32; ++w) join(m, s, red[2 * w], red[2 * w + 1], c);
        lse = m == -kInf ? (s == s ? -kInf : s) : m + a.tau * logf(s);
        float loss = 0.0f;
        for (int k = t; k < K; k += kThreads)
            if (q[k] != 0.0f) loss += q[k] * (d[k] - (xk[k] - lse));
        loss = a.tau * block_sum(loss, red);
        if (t == 0) {
            a.loss[row] = some && lse != -kInf ? loss : 0.0f;
            if (a.lse) a.lse[row] = lse;
        }
    } else {
        lse = a.lse[row];
    }
    if (PART == kDistillForward) return;
    const float g = (a.scale ? a.scale[row] : 1.0f) * a.tau;
    const bool live = some && lse != -kInf;
    T *out = static_cast<T *>(a.grad) + row * a.sg;
    __syncthreads();
    for (unsigned j = t; j < a.vocab; j += kThreads) {
        const float p = exp2f((to_f32(x[j]) - lse) * c);
        out[j] = from_f32<T>(live ? g * (S * p) : 0.0f);
    }
    __syncthreads();
    if (!live) return;
    for (int k = t; k < K; k += kThreads) {
        if (at[k] < 0) continue;
        bool first = true;
        float sum = 0.0f;
        for (int i = 0; i < K; ++i)
            if (at[i] == at[k]) {
                if (i < k) first = false;
                sum += q[i];
            }
        if (first) out[at[k]] = from_f32<T>(g * (S * exp2f((xk[k] - lse) * c) - sum));
    }
}

template <typename T>
cudaError_t launch_t(DistillPart part, const DistillArgs &a, cudaStream_t st)
{
    const unsigned grid = (unsigned)a.rows;
    if (part == kDistillForward) k_distill<T, kDistillForward><<<grid, kThreads, 0, st>>>(a);
    else if (part == kDistillBackward) k_distill<T, kDistillBackward><<<grid, kThreads, 0, st>>>(a);
    else k_distill<T, kDistillStep><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_distill(int type, DistillPart part, const DistillArgs &a, cudaStream_t st)
{
    if (type == PER_TYPE_F32) return launch_t<float>(part, a, st);
    if (type == PER_TYPE_F16) return launch_t<__half>(part, a, st);
    return launch_t<__nv_bfloat16>(part, a, st);
}

}  // namespace gbper
