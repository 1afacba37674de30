// ops_internal.cuh -- shared declarations of the learner's and the actor's operators
// (k_distill.cu, k_verify.cu, k_scan.cu; argument checks in ops_api.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gbper.h"
#include "per_internal.cuh"

namespace gbper {

constexpr uint32_t kMaxVocab = 1u << 18;   // of a distillation and of a verification

struct DistillArgs {
    const void *x, *top, *idx;
    const float *teacher_lse, *scale;
    float *loss, *lse;          // the backward pass reads lse
    void *grad;
    unsigned *status;
    long long sx, st, si, sg;   // elements between rows
    unsigned long long rows;
    unsigned vocab, k;
    int top_type;
    int idx64;
    float tau, c, c_rest;       // c + c_rest: log2(e) / tau
};

struct VerifyArgs {
    const void *p, *q, *tokens;
    const int *lens;
    const float *u, *us;
    int *accepted, *out;
    float *accept_p;
    unsigned *status;
    long long sp[2], sq[2], stok, su;
    unsigned batch, drafts, vocab;
    int tok64;
};

struct ScanArgs {
    const void *a, *x, *h, *gh;   // h: the stored states (backward)
    const float *h0, *glast;
    const uint8_t *resets;
    void *out_h, *ga, *gx;
    float *last, *gh0;
    long long sa[2], sx[2], sh[2], sgh[2], sga[2], sgx[2], sr[2];
    long long steps;
    unsigned batch, channels;
    unsigned *status;
    unsigned wait_ms;    // limit of a wait between CTAs
    unsigned withhold;   // the rank, from 1, of the CTA in each cluster that sends nothing (0: none)
};

// n / d for n < 2^31 by one multiplication: (floor(n mul / 2^32) + n) >> shift
struct FastDiv {
    unsigned d, mul, shift;
    __host__ void set(unsigned by)
    {
        d = by;
        shift = 0;
        while ((1ull << shift) < by) ++shift;
        mul = (unsigned)((((1ull << shift) - by) << 32) / by + 1);
    }
    __device__ __forceinline__ unsigned div(unsigned n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// The paged cache of a call.  Sequence b's slot s: page table[b * st + s / S], slot s mod S of it.
struct CacheArgs {
    void *k, *v;
    const int *table;
    unsigned *status;
    long long sk[3], sv[3], st;
    unsigned pages, width, heads, dim;
    FastDiv page;
    int vec;                    // every head starts on 16 bytes and ends there
};

struct AppendArgs {
    CacheArgs c;
    const void *k, *v, *q;
    void *q_out;
    const int *starts, *counts, *positions;
    const float *inv_freq;
    long long si[2][3], sq[3], sqo[3], sp;
    unsigned batch, tokens, q_heads, rot;
    int interleaved;
};

struct AttendArgs {
    CacheArgs c;
    const void *q;
    const int *lens, *counts;
    const uint8_t *mask;
    void *out;
    float *lse;
    float *work;
    long long sq[3], so[3], sm[2];
    unsigned batch, nodes, q_heads;
    float c2;                   // scale log2(e)
    int qvec, ovec;             // queries, outputs move in 16-byte pieces (outputs eight entries at a time)
    unsigned wait_ms;           // limit of a wait
    unsigned withhold;          // the barrier, from 1, that expects an arrival more than come (0: none)
};

struct KeepArgs {
    CacheArgs c;
    const int *lens, *path, *kept;
    long long sp;
    unsigned batch, nodes, most;
};

enum DistillPart { kDistillForward = 0, kDistillBackward = 1, kDistillStep = 2 };

cudaError_t launch_distill(int type, DistillPart part, const DistillArgs &a, cudaStream_t st);
cudaError_t launch_verify(int type, const VerifyArgs &a, cudaStream_t st);
cudaError_t launch_scan_forward(int type, bool sigmoid, const ScanArgs &a, cudaStream_t st);
cudaError_t launch_scan_backward(int type, bool sigmoid, const ScanArgs &a, cudaStream_t st);
cudaError_t launch_append(int type, const AppendArgs &a, cudaStream_t st);
cudaError_t launch_keep(int type, const KeepArgs &a, cudaStream_t st);
cudaError_t launch_attend(int type, const AttendArgs &a, cudaStream_t st);
cudaError_t attend_work(int type, const AttendArgs &a, unsigned long long *bytes);

// ---- element types ------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float load_typed(const void *p, long long i, int type)
{
    if (type == PER_TYPE_F32) return static_cast<const float *>(p)[i];
    if (type == PER_TYPE_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ long long load_index(const void *p, long long i, int wide)
{
    return wide ? static_cast<const long long *>(p)[i] : (long long)static_cast<const int *>(p)[i];
}

// 2^x by the special-function unit (2 ulp; a result below 2^-126 is 0)
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- pairs of binary32, two to an instruction -------------------------------------------------
struct F2 {
    float x, y;
};
__device__ __forceinline__ unsigned long long bits2(F2 v)
{
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ F2 from_bits2(unsigned long long b)
{
    F2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(b));
    return v;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from_bits2(r);
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from_bits2(r);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return from_bits2(r);
}
__device__ __forceinline__ float &at(F2 &v, int i) { return i ? v.y : v.x; }
__device__ __forceinline__ float at(const F2 &v, int i) { return i ? v.y : v.x; }

// 16 bytes of T in registers
template <typename T>
struct Pack {
    static constexpr int N = 16 / (int)sizeof(T);
    uint4 raw;
    __device__ __forceinline__ void unpack(float *f) const;
    __device__ __forceinline__ void pack(const float *f);
};

template <>
__device__ __forceinline__ void Pack<float>::unpack(float *f) const
{
    f[0] = __uint_as_float(raw.x);
    f[1] = __uint_as_float(raw.y);
    f[2] = __uint_as_float(raw.z);
    f[3] = __uint_as_float(raw.w);
}
template <>
__device__ __forceinline__ void Pack<float>::pack(const float *f)
{
    raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ void Pack<__nv_bfloat16>::unpack(float *f) const
{
    const unsigned w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // a bfloat16 is the upper half of a binary32
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <>
__device__ __forceinline__ void Pack<__nv_bfloat16>::pack(const float *f)
{
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const unsigned *>(&h);
    }
    raw = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void Pack<__half>::unpack(float *f) const
{
    const unsigned w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}
template <>
__device__ __forceinline__ void Pack<__half>::pack(const float *f)
{
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const unsigned *>(&h);
    }
    raw = make_uint4(w[0], w[1], w[2], w[3]);
}

// The 16 bytes that begin `off` bytes (a multiple of 2 below 16, the same for the whole warp) into the 32
// bytes of lo and hi.
__device__ __forceinline__ uint4 shift_bytes(uint4 lo, uint4 hi, unsigned off)
{
    unsigned w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (off & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const unsigned bits = (off & 3u) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// A launch whose grid is made of clusters of `cluster` CTAs (1: none) and which may begin while the kernel
// before it in the stream finishes (pdl_wait).
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), unsigned grid, unsigned block, unsigned cluster, size_t smem,
                            cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// The current device and its SMs.
struct DeviceInfo {
    int device, sms;
};
cudaError_t device_info(DeviceInfo *out);   // ops_api.cu

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace gbper
