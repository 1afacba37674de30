// ops_api.cu -- the C ABI of the learner's and the actor's operators: argument checks, then one launch.
// Nothing is kept between calls.
#include "ops_internal.cuh"

#include <atomic>
#include <cmath>
#include <cstdio>
#include <utility>

using namespace gbper;

namespace {

unsigned type_bytes(uint32_t type) { return type == PER_TYPE_F32 ? 4u : 2u; }

bool bad_type(uint32_t type) { return type > PER_TYPE_BF16; }

bool misaligned(const void *p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// A fixed buffer: recording a message allocates nothing and throws nothing.
thread_local char g_op_err[256] = "";

per_status fail(per_status s, const char *where, const char *what)
{
    std::snprintf(g_op_err, sizeof(g_op_err), "%s: %s", where, what);
    return s;
}

per_status refuse(const char *where, const char *what) { return fail(PER_ERR_INVALID_ARG, where, what); }

per_status done(cudaError_t e, const char *where)
{
    if (e == cudaSuccess) return PER_OK;
    cudaGetLastError();   // a refused launch is this call's error, not the next call's
    return fail(PER_ERR_CUDA, where, cudaGetErrorString(e));
}

// An output's rows must not overlap: each stride covers what lies inside it.
bool overlaps(int64_t stride, uint64_t count, uint64_t inner)
{
    if (count <= 1) return false;
    const uint64_t s = stride < 0 ? 0 - (uint64_t)stride : (uint64_t)stride;
    return s < inner;
}

// The two outer axes of an output (in either order of nesting).
bool overlaps2(const int64_t st[2], uint64_t n0, uint64_t n1, uint64_t inner)
{
    if (overlaps(st[0], n0, inner) || overlaps(st[1], n1, inner)) return true;
    if (n0 <= 1 || n1 <= 1) return false;
    const uint64_t s0 = st[0] < 0 ? 0 - (uint64_t)st[0] : (uint64_t)st[0];
    const uint64_t s1 = st[1] < 0 ? 0 - (uint64_t)st[1] : (uint64_t)st[1];
    return s0 >= s1 ? s0 < s1 * (n1 - 1) + inner : s1 < s0 * (n0 - 1) + inner;
}

per_status distill(const char *where, DistillPart part, const per_distill_shape *sh, const void *x, const void *top,
                   const void *idx, const float *tlse, const float *scale, float *loss, float *lse, void *grad,
                   uint32_t *status, void *stream)
{
    if (!sh) return refuse(where, "shape is NULL");
    if (sh->rows > 0x7fffffffull) return refuse(where, "rows must be below 2^31");
    if (sh->vocab == 0 || sh->vocab > kMaxVocab) return refuse(where, "vocab must be in 1 .. 2^18");
    if (sh->top == 0 || sh->top > 1024) return refuse(where, "top must be in 1 .. 1024");
    if (bad_type(sh->type) || bad_type(sh->top_type)) return refuse(where, "unknown element type");
    if (sh->flags & ~(uint32_t)PER_DISTILL_IDX64) return refuse(where, "unknown flags");
    if (!(sh->temperature > 0.0f) || !std::isfinite(sh->temperature) || !std::isfinite(1.5f / sh->temperature))
        return refuse(where, "temperature must be finite and > 0");
    if (sh->rows == 0) return PER_OK;
    if (!x || !top || !idx) return refuse(where, "logits, top and idx are required");
    if (part != kDistillBackward && !loss) return refuse(where, "loss is required");
    if (part == kDistillBackward && !lse) return refuse(where, "lse is required");
    if (part != kDistillForward && !grad) return refuse(where, "grad is required");
    const unsigned e = type_bytes(sh->type);
    if (misaligned(x, e) || misaligned(grad, e) || misaligned(top, type_bytes(sh->top_type)) ||
        misaligned(idx, sh->flags & PER_DISTILL_IDX64 ? 8 : 4) || misaligned(tlse, 4) || misaligned(scale, 4) ||
        misaligned(loss, 4) || misaligned(lse, 4) || misaligned(status, 4))
        return refuse(where, "misaligned pointer");
    if (part != kDistillForward && overlaps(sh->stride_grad, sh->rows, sh->vocab))
        return refuse(where, "rows of grad overlap");
    if (part != kDistillForward && grad == x && sh->stride_grad != sh->stride_logits)
        return refuse(where, "grad in the place of logits needs their stride");
    DistillArgs a{};
    a.x = x;
    a.top = top;
    a.idx = idx;
    a.teacher_lse = tlse;
    a.scale = scale;
    a.loss = loss;
    a.lse = lse;
    a.grad = grad;
    a.status = status;
    a.sx = sh->stride_logits;
    a.st = sh->stride_top;
    a.si = sh->stride_idx;
    a.sg = sh->stride_grad;
    a.rows = sh->rows;
    a.vocab = sh->vocab;
    a.k = sh->top;
    a.top_type = (int)sh->top_type;
    a.idx64 = (sh->flags & PER_DISTILL_IDX64) != 0;
    a.tau = sh->temperature;
    const double c = 1.4426950408889634 / (double)sh->temperature;
    a.c = (float)c;
    a.c_rest = (float)(c - (double)a.c);
    return done(launch_distill((int)sh->type, part, a, reinterpret_cast<cudaStream_t>(stream)), where);
}

// What both directions of the scan check; 1: nothing to launch.
per_status scan_check(const char *where, const per_scan_shape *sh, bool *empty)
{
    if (!sh) return refuse(where, "shape is NULL");
    if (sh->steps > 0x7fffffffull) return refuse(where, "steps must be below 2^31");
    if ((uint64_t)sh->batch * sh->channels > 0x7fffffffull) return refuse(where, "batch x channels must be below 2^31");
    if (bad_type(sh->type)) return refuse(where, "unknown element type");
    if (sh->flags & ~(uint32_t)(PER_SCAN_SIGMOID | PER_SCAN_REVERSE)) return refuse(where, "unknown flags");
    if (sh->wait_limit_ms > 10000) return refuse(where, "wait_limit_ms must be at most 10000");
    if (sh->withhold > 16) return refuse(where, "withhold must be at most 16");
    if (misaligned(sh->d_status, 4)) return refuse(where, "misaligned pointer");
    *empty = sh->batch == 0 || sh->channels == 0;
    return PER_OK;
}

void set_waits(ScanArgs &a, const per_scan_shape *sh)
{
    a.status = sh->d_status;
    a.wait_ms = sh->wait_limit_ms ? sh->wait_limit_ms : 2000;
    a.withhold = sh->withhold;
}

// Moves an array's start to the first step that the pass takes and turns its time axis.
template <typename P>
void set_axis(P **p, const void *src, const int64_t stride[2], long long dst[2], const per_scan_shape *sh, unsigned bytes)
{
    dst[0] = stride[0];
    dst[1] = stride[1];
    const char *c = static_cast<const char *>(src);
    if (c && (sh->flags & PER_SCAN_REVERSE) && sh->steps) {
        c += (int64_t)(sh->steps - 1) * stride[1] * (int64_t)bytes;
        dst[1] = -stride[1];
    }
    *p = reinterpret_cast<P *>(const_cast<char *>(c));
}

// ---- the paged cache ------------------------------------------------------------------------

const char *cache_fault(const per_cache &c)
{
    if (c.pages > 0x7fffffffu) return "pages must be below 2^31";
    if (c.page == 0 || c.page > (1u << 20)) return "page must be in 1 .. 2^20";
    if ((uint64_t)c.width * c.page > 1ull << 30) return "width x page must be at most 2^30";
    if (c.heads == 0 || c.heads > 4096) return "heads must be in 1 .. 4096";
    if (c.dim == 0 || c.dim > 256) return "dim must be in 1 .. 256";
    if (bad_type(c.type)) return "unknown element type";
    return nullptr;
}

bool on16(const void *p, const int64_t *stride, int n, unsigned e)
{
    if (misaligned(p, 16)) return false;
    for (int i = 0; i < n; ++i)
        if (stride[i] * (int64_t)e % 16 != 0) return false;
    return true;
}

CacheArgs cache_args(const per_cache &c, void *k, void *v, const int32_t *table, uint32_t *status)
{
    CacheArgs a{};
    a.k = k;
    a.v = v;
    a.table = table;
    a.status = status;
    for (int i = 0; i < 3; ++i) {
        a.sk[i] = c.stride_k[i];
        a.sv[i] = c.stride_v[i];
    }
    a.st = c.stride_table;
    a.pages = c.pages;
    a.width = c.width;
    a.heads = c.heads;
    a.dim = c.dim;
    a.page.set(c.page);
    const unsigned e = type_bytes(c.type);
    a.vec = c.dim * e % 16 == 0 && on16(k, c.stride_k, 3, e) && on16(v, c.stride_v, 3, e);
    return a;
}

// The rows of a cache that is written to must not overlap; its three outer axes may be nested in any order.
bool overlaps3(const int64_t st[3], uint64_t n0, uint64_t n1, uint64_t n2, uint64_t inner)
{
    struct Axis {
        uint64_t s, n;
    } x[3] = {{0, n0}, {0, n1}, {0, n2}};
    for (int i = 0; i < 3; ++i) x[i].s = st[i] < 0 ? 0 - (uint64_t)st[i] : (uint64_t)st[i];
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (x[j].s > x[j + 1].s) std::swap(x[j], x[j + 1]);
    uint64_t covered = inner;   // what lies below the axis, in elements
    for (const Axis &a : x) {
        if (a.n == 0) return false;
        if (a.n == 1) continue;
        if (a.s < covered) return true;
        covered += a.s * (a.n - 1);
    }
    return false;
}

const char *attend_fault(const per_attend_shape *sh)
{
    if (!sh) return "shape is NULL";
    if (const char *f = cache_fault(sh->cache)) return f;
    if (sh->batch > (1u << 20)) return "batch must be at most 2^20";
    if (sh->nodes > 1024) return "nodes must be at most 1024";
    if (sh->q_heads == 0 || sh->q_heads % sh->cache.heads || sh->q_heads / sh->cache.heads > 64)
        return "q_heads must be 1 .. 64 times heads";
    // tiles of 32 keys, and what each sequence counts beside them
    if (((uint64_t)sh->cache.width * sh->cache.page / 32 + 3) * sh->batch * sh->cache.heads >> 45)
        return "batch x width x page x heads must be below 2^50";
    if (!std::isfinite(sh->scale) || !std::isfinite(sh->scale * 1.5f)) return "scale must be finite";
    if (sh->wait_limit_ms > 10000) return "wait_limit_ms must be at most 10000";
    if (sh->withhold > 8) return "withhold must be at most 8";
    return nullptr;
}

}  // namespace

namespace gbper {

cudaError_t device_info(DeviceInfo *out)
{
    static std::atomic<int> sms[64];   // zero: not asked yet
    cudaError_t e = cudaGetDevice(&out->device);
    if (e != cudaSuccess) return e;
    if (out->device < 0 || out->device >= 64) return cudaErrorInvalidDevice;
    out->sms = sms[out->device].load(std::memory_order_relaxed);
    if (out->sms == 0) {
        e = cudaDeviceGetAttribute(&out->sms, cudaDevAttrMultiProcessorCount, out->device);
        if (e != cudaSuccess) return e;
        sms[out->device].store(out->sms, std::memory_order_relaxed);
    }
    return cudaSuccess;
}

}  // namespace gbper

extern "C" {

const char *per_last_op_error(void) { return g_op_err; }

per_status per_distill_forward(const per_distill_shape *shape, const void *d_logits, const void *d_top,
                               const void *d_idx, const float *d_teacher_lse, float *d_loss, float *d_lse,
                               uint32_t *d_status, void *stream)
{
    return distill("per_distill_forward", kDistillForward, shape, d_logits, d_top, d_idx, d_teacher_lse, nullptr,
                   d_loss, d_lse, nullptr, d_status, stream);
}

per_status per_distill_backward(const per_distill_shape *shape, const void *d_logits, const void *d_top,
                                const void *d_idx, const float *d_teacher_lse, const float *d_lse,
                                const float *d_scale, void *d_grad, uint32_t *d_status, void *stream)
{
    return distill("per_distill_backward", kDistillBackward, shape, d_logits, d_top, d_idx, d_teacher_lse, d_scale,
                   nullptr, const_cast<float *>(d_lse), d_grad, d_status, stream);
}

per_status per_distill_step(const per_distill_shape *shape, const void *d_logits, const void *d_top, const void *d_idx,
                            const float *d_teacher_lse, const float *d_scale, float *d_loss, float *d_lse,
                            void *d_grad, uint32_t *d_status, void *stream)
{
    return distill("per_distill_step", kDistillStep, shape, d_logits, d_top, d_idx, d_teacher_lse, d_scale, d_loss,
                   d_lse, d_grad, d_status, stream);
}

per_status per_verify_draft(const per_verify_shape *shape, const void *d_p, const void *d_q, const void *d_tokens,
                            const int32_t *d_lens, const float *d_accept_u, const float *d_sample_u,
                            int32_t *d_accepted, int32_t *d_out, float *d_accept_p, uint32_t *d_status, void *stream)
{
    const char *where = "per_verify_draft";
    const per_verify_shape *sh = shape;
    if (!sh) return refuse(where, "shape is NULL");
    if (sh->batch > (1u << 20)) return refuse(where, "batch must be at most 2^20");
    if (sh->drafts > 1024) return refuse(where, "drafts must be at most 1024");
    if (sh->vocab == 0 || sh->vocab > kMaxVocab) return refuse(where, "vocab must be in 1 .. 2^18");
    if (bad_type(sh->type)) return refuse(where, "unknown element type");
    if ((sh->flags & ~(uint32_t)PER_VERIFY_TOKENS64) || sh->reserved) return refuse(where, "unknown flags");
    if (sh->batch == 0) return PER_OK;
    if (!d_p || !d_sample_u || !d_accepted || !d_out) return refuse(where, "p, sample_u, accepted and out are required");
    if (sh->drafts && (!d_tokens || !d_accept_u)) return refuse(where, "tokens and accept_u are required");
    const unsigned e = type_bytes(sh->type);
    if (misaligned(d_p, e) || misaligned(d_q, e) || misaligned(d_tokens, sh->flags & PER_VERIFY_TOKENS64 ? 8 : 4) ||
        misaligned(d_lens, 4) || misaligned(d_accept_u, 4) || misaligned(d_sample_u, 4) || misaligned(d_accepted, 4) ||
        misaligned(d_out, 4) || misaligned(d_accept_p, 4) || misaligned(d_status, 4))
        return refuse(where, "misaligned pointer");
    VerifyArgs a{};
    a.p = d_p;
    a.q = sh->drafts ? d_q : nullptr;
    a.tokens = d_tokens;
    a.lens = d_lens;
    a.u = d_accept_u;
    a.us = d_sample_u;
    a.accepted = d_accepted;
    a.out = d_out;
    a.accept_p = d_accept_p;
    a.status = d_status;
    for (int i = 0; i < 2; ++i) {
        a.sp[i] = sh->stride_p[i];
        a.sq[i] = sh->stride_q[i];
    }
    a.stok = sh->stride_tokens;
    a.su = sh->stride_u;
    a.batch = sh->batch;
    a.drafts = sh->drafts;
    a.vocab = sh->vocab;
    a.tok64 = (sh->flags & PER_VERIFY_TOKENS64) != 0;
    return done(launch_verify((int)sh->type, a, reinterpret_cast<cudaStream_t>(stream)), where);
}

per_status per_scan_forward(const per_scan_shape *shape, const void *d_a, const void *d_x, const float *d_h0,
                            const uint8_t *d_resets, void *d_h, float *d_last, void *stream)
{
    const char *where = "per_scan_forward";
    bool empty = false;
    const per_status s = scan_check(where, shape, &empty);
    if (s != PER_OK || empty) return s;
    const unsigned e = type_bytes(shape->type);
    if (shape->steps && (!d_a || !d_x || !d_h)) return refuse(where, "a, x and h are required");
    if (misaligned(d_a, e) || misaligned(d_x, e) || misaligned(d_h, e) || misaligned(d_h0, 4) || misaligned(d_last, 4))
        return refuse(where, "misaligned pointer");
    if (overlaps2(shape->stride_h, shape->batch, shape->steps, shape->channels)) return refuse(where, "rows of h overlap");
    ScanArgs a{};
    set_axis(&a.a, d_a, shape->stride_a, a.sa, shape, e);
    set_axis(&a.x, d_x, shape->stride_x, a.sx, shape, e);
    set_axis(&a.out_h, d_h, shape->stride_h, a.sh, shape, e);
    set_axis(&a.resets, d_resets, shape->stride_resets, a.sr, shape, 1);
    a.h0 = d_h0;
    a.last = d_last;
    a.steps = (long long)shape->steps;
    a.batch = shape->batch;
    a.channels = shape->channels;
    set_waits(a, shape);
    return done(launch_scan_forward((int)shape->type, (shape->flags & PER_SCAN_SIGMOID) != 0, a,
                                    reinterpret_cast<cudaStream_t>(stream)), where);
}

per_status per_scan_backward(const per_scan_shape *shape, const void *d_a, const void *d_x, const void *d_h,
                             const float *d_h0, const uint8_t *d_resets, const void *d_gh, const float *d_glast,
                             void *d_ga, void *d_gx, float *d_gh0, void *stream)
{
    const char *where = "per_scan_backward";
    bool empty = false;
    const per_status s = scan_check(where, shape, &empty);
    if (s != PER_OK || empty) return s;
    const unsigned e = type_bytes(shape->type);
    const bool sig = (shape->flags & PER_SCAN_SIGMOID) != 0;
    if (shape->steps && (!d_a || !d_h || !d_gh)) return refuse(where, "a, h and gh are required");
    if (shape->steps && sig && !d_x) return refuse(where, "x is required with a sigmoid gate");
    if (misaligned(d_a, e) || misaligned(d_x, e) || misaligned(d_h, e) || misaligned(d_gh, e) || misaligned(d_ga, e) ||
        misaligned(d_gx, e) || misaligned(d_h0, 4) || misaligned(d_glast, 4) || misaligned(d_gh0, 4))
        return refuse(where, "misaligned pointer");
    if ((d_ga && overlaps2(shape->stride_ga, shape->batch, shape->steps, shape->channels)) ||
        (d_gx && overlaps2(shape->stride_gx, shape->batch, shape->steps, shape->channels)))
        return refuse(where, "rows of a gradient overlap");
    ScanArgs a{};
    set_axis(&a.a, d_a, shape->stride_a, a.sa, shape, e);
    set_axis(&a.x, sig ? d_x : nullptr, shape->stride_x, a.sx, shape, e);
    set_axis(&a.h, d_h, shape->stride_h, a.sh, shape, e);
    set_axis(&a.gh, d_gh, shape->stride_gh, a.sgh, shape, e);
    set_axis(&a.ga, d_ga, shape->stride_ga, a.sga, shape, e);
    set_axis(&a.gx, d_gx, shape->stride_gx, a.sgx, shape, e);
    set_axis(&a.resets, d_resets, shape->stride_resets, a.sr, shape, 1);
    a.h0 = d_h0;
    a.glast = d_glast;
    a.gh0 = d_gh0;
    a.steps = (long long)shape->steps;
    a.batch = shape->batch;
    a.channels = shape->channels;
    set_waits(a, shape);
    return done(launch_scan_backward((int)shape->type, sig, a, reinterpret_cast<cudaStream_t>(stream)), where);
}

per_status per_cache_append(const per_append_shape *shape, const void *d_k, const void *d_v, const void *d_q,
                            void *d_k_cache, void *d_v_cache, void *d_q_out, const int32_t *d_table,
                            const int32_t *d_starts, const int32_t *d_counts, const int32_t *d_positions,
                            const float *d_inv_freq, uint32_t *d_status, void *stream)
{
    const char *where = "per_cache_append";
    const per_append_shape *sh = shape;
    if (!sh) return refuse(where, "shape is NULL");
    const per_cache &c = sh->cache;
    if (const char *f = cache_fault(c)) return refuse(where, f);
    if (sh->batch > (1u << 20)) return refuse(where, "batch must be at most 2^20");
    if ((uint64_t)sh->batch * sh->tokens > 0x7fffffffull) return refuse(where, "batch x tokens must be below 2^31");
    if (sh->q_heads > 4096) return refuse(where, "q_heads must be at most 4096");
    if (sh->rot > c.dim || sh->rot % 2) return refuse(where, "rot must be even and at most dim");
    if ((sh->flags & ~(uint32_t)PER_APPEND_INTERLEAVED) || sh->reserved) return refuse(where, "unknown flags");
    if (sh->batch == 0 || sh->tokens == 0) return PER_OK;
    if (!d_k || !d_v || !d_starts) return refuse(where, "k, v and starts are required");
    if (c.pages && (!d_k_cache || !d_v_cache)) return refuse(where, "the caches are required");
    if (c.width && !d_table) return refuse(where, "table is required");
    if (sh->q_heads && (!d_q || !d_q_out)) return refuse(where, "q and q_out are required");
    if (sh->rot && !d_inv_freq) return refuse(where, "inv_freq is required");
    const unsigned e = type_bytes(c.type);
    if (misaligned(d_k, e) || misaligned(d_v, e) || misaligned(d_q, e) || misaligned(d_q_out, e) ||
        misaligned(d_k_cache, e) || misaligned(d_v_cache, e) || misaligned(d_table, 4) || misaligned(d_starts, 4) ||
        misaligned(d_counts, 4) || misaligned(d_positions, 4) || misaligned(d_inv_freq, 4) || misaligned(d_status, 4))
        return refuse(where, "misaligned pointer");
    if (overlaps3(c.stride_k, c.pages, c.page, c.heads, c.dim) || overlaps3(c.stride_v, c.pages, c.page, c.heads, c.dim))
        return refuse(where, "rows of a cache overlap");
    if (sh->q_heads && overlaps3(sh->stride_q_out, sh->batch, sh->tokens, sh->q_heads, c.dim))
        return refuse(where, "rows of q_out overlap");
    if (sh->q_heads && d_q == d_q_out)
        for (int i = 0; i < 3; ++i)
            if (sh->stride_q[i] != sh->stride_q_out[i]) return refuse(where, "q_out in the place of q needs its strides");
    if (c.pages && d_k_cache == d_v_cache) return refuse(where, "keys and values in the same memory");
    AppendArgs a{};
    a.c = cache_args(c, d_k_cache, d_v_cache, d_table, d_status);
    a.k = d_k;
    a.v = d_v;
    a.q = d_q;
    a.q_out = d_q_out;
    a.starts = d_starts;
    a.counts = d_counts;
    a.positions = d_positions;
    a.inv_freq = d_inv_freq;
    for (int i = 0; i < 3; ++i) {
        a.si[0][i] = sh->stride_in[0][i];
        a.si[1][i] = sh->stride_in[1][i];
        a.sq[i] = sh->stride_q[i];
        a.sqo[i] = sh->stride_q_out[i];
    }
    a.sp = sh->stride_positions;
    a.batch = sh->batch;
    a.tokens = sh->tokens;
    a.q_heads = sh->q_heads;
    a.rot = sh->rot;
    a.interleaved = (sh->flags & PER_APPEND_INTERLEAVED) != 0;
    // whole 16-byte pieces everywhere, and a rotation that begins and ends with one
    a.c.vec = a.c.vec && on16(d_k, sh->stride_in[0], 3, e) && on16(d_v, sh->stride_in[1], 3, e) &&
              (!sh->q_heads || (on16(d_q, sh->stride_q, 3, e) && on16(d_q_out, sh->stride_q_out, 3, e))) &&
              sh->rot * e % (a.interleaved ? 16 : 32) == 0;
    return done(launch_append((int)c.type, a, reinterpret_cast<cudaStream_t>(stream)), where);
}

per_status per_tree_attention_work(const per_attend_shape *shape, const void *d_k_cache, const void *d_v_cache,
                                   uint64_t *bytes)
{
    const char *where = "per_tree_attention_work";
    if (const char *f = attend_fault(shape)) return refuse(where, f);
    if (!bytes) return refuse(where, "bytes is NULL");
    *bytes = 0;
    if (shape->batch == 0 || shape->nodes == 0) return PER_OK;
    AttendArgs a{};
    a.c = cache_args(shape->cache, const_cast<void *>(d_k_cache), const_cast<void *>(d_v_cache), nullptr, nullptr);
    a.batch = shape->batch;
    a.nodes = shape->nodes;
    a.q_heads = shape->q_heads;
    a.c2 = (float)((double)shape->scale * 1.4426950408889634);
    unsigned long long n = 0;
    const cudaError_t e = attend_work((int)shape->cache.type, a, &n);
    *bytes = n;
    return done(e, where);
}

per_status per_tree_attention(const per_attend_shape *shape, const void *d_q, const void *d_k_cache,
                              const void *d_v_cache, const int32_t *d_table, const int32_t *d_lens,
                              const int32_t *d_counts, const uint8_t *d_mask, void *d_out, float *d_lse,
                              void *d_work, uint32_t *d_status, void *stream)
{
    const char *where = "per_tree_attention";
    if (const char *f = attend_fault(shape)) return refuse(where, f);
    const per_cache &c = shape->cache;
    if (shape->batch == 0 || shape->nodes == 0) return PER_OK;
    if (!d_q || !d_lens || !d_out) return refuse(where, "q, lens and out are required");
    if (c.pages && (!d_k_cache || !d_v_cache)) return refuse(where, "the caches are required");
    if (c.width && !d_table) return refuse(where, "table is required");
    const unsigned e = type_bytes(c.type);
    if (misaligned(d_q, e) || misaligned(d_k_cache, e) || misaligned(d_v_cache, e) || misaligned(d_out, e) ||
        misaligned(d_table, 4) || misaligned(d_lens, 4) || misaligned(d_counts, 4) || misaligned(d_lse, 4) ||
        misaligned(d_work, 16) || misaligned(d_status, 4))
        return refuse(where, "misaligned pointer");
    if (overlaps3(shape->stride_out, shape->batch, shape->nodes, shape->q_heads, c.dim))
        return refuse(where, "rows of out overlap");
    AttendArgs a{};
    a.c = cache_args(c, const_cast<void *>(d_k_cache), const_cast<void *>(d_v_cache), d_table, d_status);
    a.q = d_q;
    a.lens = d_lens;
    a.counts = d_counts;
    a.mask = d_mask;
    a.out = d_out;
    a.lse = d_lse;
    a.work = static_cast<float *>(d_work);
    for (int i = 0; i < 3; ++i) {
        a.sq[i] = shape->stride_q[i];
        a.so[i] = shape->stride_out[i];
    }
    a.sm[0] = shape->stride_mask[0];
    a.sm[1] = shape->stride_mask[1];
    a.batch = shape->batch;
    a.nodes = shape->nodes;
    a.q_heads = shape->q_heads;
    a.c2 = (float)((double)shape->scale * 1.4426950408889634);
    a.qvec = c.dim * e % 16 == 0 && on16(d_q, shape->stride_q, 3, e);
    a.wait_ms = shape->wait_limit_ms ? shape->wait_limit_ms : 2000;
    a.withhold = shape->withhold;
    a.ovec = c.dim % 8 == 0 && on16(d_out, shape->stride_out, 3, e);
    unsigned long long need = 0;
    const cudaError_t err = attend_work((int)c.type, a, &need);
    if (err != cudaSuccess) return done(err, where);
    if (need > shape->work_bytes || (need && !d_work)) return refuse(where, "work is smaller than per_tree_attention_work says");
    return done(launch_attend((int)c.type, a, reinterpret_cast<cudaStream_t>(stream)), where);
}

per_status per_cache_keep(const per_keep_shape *shape, void *d_k_cache, void *d_v_cache, const int32_t *d_table,
                          const int32_t *d_lens, const int32_t *d_path, const int32_t *d_kept, uint32_t *d_status,
                          void *stream)
{
    const char *where = "per_cache_keep";
    const per_keep_shape *sh = shape;
    if (!sh) return refuse(where, "shape is NULL");
    const per_cache &c = sh->cache;
    if (const char *f = cache_fault(c)) return refuse(where, f);
    if (sh->batch > (1u << 20)) return refuse(where, "batch must be at most 2^20");
    if (sh->nodes > (1u << 20)) return refuse(where, "nodes must be at most 2^20");
    if (sh->most > 1024) return refuse(where, "most must be at most 1024");
    if (sh->reserved) return refuse(where, "unknown flags");
    if (sh->batch == 0 || sh->most == 0) return PER_OK;
    if (!d_lens || !d_path || !d_kept) return refuse(where, "lens, path and kept are required");
    if (c.pages && (!d_k_cache || !d_v_cache)) return refuse(where, "the caches are required");
    if (c.width && !d_table) return refuse(where, "table is required");
    const unsigned e = type_bytes(c.type);
    if (misaligned(d_k_cache, e) || misaligned(d_v_cache, e) || misaligned(d_table, 4) || misaligned(d_lens, 4) ||
        misaligned(d_path, 4) || misaligned(d_kept, 4) || misaligned(d_status, 4))
        return refuse(where, "misaligned pointer");
    if (overlaps3(c.stride_k, c.pages, c.page, c.heads, c.dim) || overlaps3(c.stride_v, c.pages, c.page, c.heads, c.dim))
        return refuse(where, "rows of a cache overlap");
    if (c.pages && d_k_cache == d_v_cache) return refuse(where, "keys and values in the same memory");
    KeepArgs a{};
    a.c = cache_args(c, d_k_cache, d_v_cache, d_table, d_status);
    a.lens = d_lens;
    a.path = d_path;
    a.kept = d_kept;
    a.sp = sh->stride_path;
    a.batch = sh->batch;
    a.nodes = sh->nodes;
    a.most = sh->most;
    return done(launch_keep((int)c.type, a, reinterpret_cast<cudaStream_t>(stream)), where);
}

}  // extern "C"
