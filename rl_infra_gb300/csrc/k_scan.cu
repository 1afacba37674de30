// k_scan.cu -- the gated linear recurrence and its gradient: one thread takes one channel of one
// sequence through time.
#include "ops_internal.cuh"

namespace gbper {

namespace {

constexpr int kThreads = 128;

struct Gate {
    float w, v;   // the state's weight and the input's
};

template <bool SIG>
__device__ __forceinline__ Gate gate(float a)
{
    if (!SIG) return {a, 1.0f};
    const float e = expf(-fabsf(a)), r = 1.0f / (1.0f + e);
    return a >= 0.0f ? Gate{r, e * r} : Gate{e * r, r};
}

// w h with a weight of 0 dropping whatever h holds
__device__ __forceinline__ float weigh(float w, float h, float more) { return w == 0.0f ? more : fmaf(w, h, more); }

template <typename T, bool SIG>
__global__ void __launch_bounds__(kThreads) k_scan_fwd(ScanArgs s)
{
    const unsigned blocks = (s.channels + kThreads - 1) / kThreads;
    const unsigned c = blockIdx.x % blocks * kThreads + threadIdx.x;
    if (c >= s.channels) return;
    const long long b = blockIdx.x / blocks;
    const T *a = static_cast<const T *>(s.a) + b * s.sa[0] + c;
    const T *x = static_cast<const T *>(s.x) + b * s.sx[0] + c;
    T *o = static_cast<T *>(s.out_h) + b * s.sh[0] + c;
    float h = s.h0 ? s.h0[b * s.channels + c] : 0.0f;
    for (long long t = 0; t < s.steps; ++t) {
        const Gate g = gate<SIG>(to_f32(a[t * s.sa[1]]));
        const bool reset = s.resets && s.resets[b * s.sr[0] + t * s.sr[1]];
        const float in = to_f32(x[t * s.sx[1]]);
        h = weigh(reset ? 0.0f : g.w, h, SIG ? weigh(g.v, in, 0.0f) : in);
        o[t * s.sh[1]] = from_f32<T>(h);
    }
    if (s.last) s.last[b * s.channels + c] = h;
}

template <typename T, bool SIG>
__global__ void __launch_bounds__(kThreads) k_scan_bwd(ScanArgs s)
{
    const unsigned blocks = (s.channels + kThreads - 1) / kThreads;
    const unsigned c = blockIdx.x % blocks * kThreads + threadIdx.x;
    if (c >= s.channels) return;
    const long long b = blockIdx.x / blocks;
    const T *a = static_cast<const T *>(s.a) + b * s.sa[0] + c;
    const T *x = static_cast<const T *>(s.x) + b * s.sx[0] + c;
    const T *h = static_cast<const T *>(s.h) + b * s.sh[0] + c;
    const T *gh = static_cast<const T *>(s.gh) + b * s.sgh[0] + c;
    T *ga = s.ga ? static_cast<T *>(s.ga) + b * s.sga[0] + c : nullptr;
    T *gx = s.gx ? static_cast<T *>(s.gx) + b * s.sgx[0] + c : nullptr;
    float carry = s.glast ? s.glast[b * s.channels + c] : 0.0f;
    const float h0 = s.h0 ? s.h0[b * s.channels + c] : 0.0f;
    for (long long t = s.steps - 1; t >= 0; --t) {
        const Gate w = gate<SIG>(to_f32(a[t * s.sa[1]]));
        const bool reset = s.resets && s.resets[b * s.sr[0] + t * s.sr[1]];
        const float g = to_f32(gh[t * s.sgh[1]]) + carry;
        const float before = reset ? 0.0f : t ? to_f32(h[(t - 1) * s.sh[1]]) : h0;
        if (SIG) {
            const float ww = w.w * w.v;
            if (ga) ga[t * s.sga[1]] = from_f32<T>(ww == 0.0f ? 0.0f : g * (before - to_f32(x[t * s.sx[1]])) * ww);
            if (gx) gx[t * s.sgx[1]] = from_f32<T>(weigh(w.v, g, 0.0f));
        } else {
            if (ga) ga[t * s.sga[1]] = from_f32<T>(reset ? 0.0f : g * before);
            if (gx) gx[t * s.sgx[1]] = from_f32<T>(g);
        }
        carry = weigh(reset ? 0.0f : w.w, g, 0.0f);
    }
    if (s.gh0) s.gh0[b * s.channels + c] = carry;
}

template <typename T>
cudaError_t fwd_t(bool sig, const ScanArgs &a, cudaStream_t st)
{
    const unsigned grid = (a.channels + kThreads - 1) / kThreads * a.batch;
    if (sig) k_scan_fwd<T, true><<<grid, kThreads, 0, st>>>(a);
    else k_scan_fwd<T, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(bool sig, const ScanArgs &a, cudaStream_t st)
{
    const unsigned grid = (a.channels + kThreads - 1) / kThreads * a.batch;
    if (sig) k_scan_bwd<T, true><<<grid, kThreads, 0, st>>>(a);
    else k_scan_bwd<T, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_forward(int type, bool sigmoid, const ScanArgs &a, cudaStream_t st)
{
    if (type == PER_TYPE_F32) return fwd_t<float>(sigmoid, a, st);
    if (type == PER_TYPE_F16) return fwd_t<__half>(sigmoid, a, st);
    return fwd_t<__nv_bfloat16>(sigmoid, a, st);
}

cudaError_t launch_scan_backward(int type, bool sigmoid, const ScanArgs &a, cudaStream_t st)
{
    if (type == PER_TYPE_F32) return bwd_t<float>(sigmoid, a, st);
    if (type == PER_TYPE_F16) return bwd_t<__half>(sigmoid, a, st);
    return bwd_t<__nv_bfloat16>(sigmoid, a, st);
}

}  // namespace gbper
