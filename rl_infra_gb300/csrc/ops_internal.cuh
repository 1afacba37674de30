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
    float tau;
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
};

enum DistillPart { kDistillForward = 0, kDistillBackward = 1, kDistillStep = 2 };

cudaError_t launch_distill(int type, DistillPart part, const DistillArgs &a, cudaStream_t st);
cudaError_t launch_verify(int type, const VerifyArgs &a, cudaStream_t st);
cudaError_t launch_scan_forward(int type, bool sigmoid, const ScanArgs &a, cudaStream_t st);
cudaError_t launch_scan_backward(int type, bool sigmoid, const ScanArgs &a, cudaStream_t st);

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

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

}  // namespace gbper
