// k_cache.cu -- writing to a paged cache: new keys and values with the position rotation on the way, and
// the move of a tree's accepted path.
//
// Append.  Every byte of k, v and q is read once and written once: HBM bounds long prompts, the launch and
// a chain of three loads (table, row, frequency) bounds a single token.  A CTA takes a few tokens.  It first
// works out their cosines and sines (once for all heads) and the addresses of their slots into
// shared memory, then its threads move the heads in pieces of two times 16 bytes: the two halves that turn
// together, or two neighbouring pieces of what is copied.
//
// The angle pos * f is needed modulo one turn.  f / 2 pi is taken as a 64-bit fraction of a turn (the
// 24-bit mantissa times the first 64 bits of 1 / 2 pi), so that pos times it modulo 2^64 is the reduced
// angle to 2^-64 pos, in integers: no binary64, of which an SM retires a warp's instruction in 16 cycles.
//
// Measured (GB300): four prompts of 8191 tokens, 32 + 8 + 8 heads of 128 entries, bf16 117 us, 6.0 TB/s (90% of the copy
// rate); 64 trees of 24 nodes, f16 12.7 us from HBM, 10.3 from L2 (floor 5.3: the heads are asked for only when places and
// angles stand); one token 3.0 us.
//
// Keep.  A thread owns 16 bytes of a head and moves them along the path.  Since path_j >= j grows, a slot
// is read before or in the same batch of loads as anything is written to it.  1024 paths of up to 12 nodes, 8 heads of
// 128 binary32 entries 19.2 us from HBM (109 MB, 85% of the copy rate; 13.3 us from L2); 64 of up to 6, bf16 2.4 us.
#include "ops_internal.cuh"

#include <algorithm>

namespace gbper {

namespace {

typedef unsigned long long u64;
constexpr int kThreads = 256;
constexpr unsigned kMaxTokens = 32;   // tokens of a CTA

// f / (2 pi) in units of 2^-64, modulo 2^64
__device__ __forceinline__ u64 turns(float f)
{
    constexpr u64 kInv2Pi = 0x28be60db9391054aull;   // floor(2^64 / (2 pi))
    const unsigned b = __float_as_uint(f);
    const unsigned e = (b >> 23) & 0xffu;
    const u64 m = e ? (b & 0x7fffffu) | 0x800000u : (b & 0x7fffffu);
    const int s = 150 - (int)(e ? e : 1);            // |f| = m 2^-s
    const u64 lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    u64 w;
    if (s >= 128) w = 0;
    else if (s >= 64) w = s == 64 ? hi : hi >> (s - 64);
    else if (s > 0) w = (hi << (64 - s)) | (lo >> s);
    else w = s > -64 ? lo << -s : 0;
    return b >> 31 ? 0 - w : w;
}

__device__ __forceinline__ float2 cos_sin(float f, int pos)
{
    if ((__float_as_uint(f) & 0x7f800000u) == 0x7f800000u) return make_float2(NAN, NAN);
    const u64 phase = turns(f) * (u64)(long long)pos;
    float s, c;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c, s);
}

// N elements of T as they lie in memory
template <typename T, int N> struct Piece;
template <typename T> struct Piece<T, 1> {
    T raw;
    __device__ __forceinline__ void get(float *f) const { f[0] = to_f32(raw); }
    __device__ __forceinline__ void set(const float *f) { raw = from_f32<T>(f[0]); }
    __device__ __forceinline__ void zero() { raw = from_f32<T>(0.0f); }
};
template <typename T, int N> struct Piece {
    Pack<T> p;
    __device__ __forceinline__ void get(float *f) const { p.unpack(f); }
    __device__ __forceinline__ void set(const float *f) { p.pack(f); }
    __device__ __forceinline__ void zero() { p.raw = make_uint4(0, 0, 0, 0); }
};
template <typename T, int N>
__device__ __forceinline__ Piece<T, N> load_piece(const T *p)
{
    Piece<T, N> r;
    if constexpr (N == 1) r.raw = *p;
    else r.p.raw = *reinterpret_cast<const uint4 *>(p);
    return r;
}
template <typename T, int N>
__device__ __forceinline__ void store_piece(T *p, const Piece<T, N> &r)
{
    if constexpr (N == 1) *p = r.raw;
    else *reinterpret_cast<uint4 *>(p) = r.p.raw;
}

// The element offset of slot `s` of a sequence in the keys and in the values; false if it has no page.
__device__ __forceinline__ bool place(const CacheArgs &c, long long b, long long s, long long *ok, long long *ov)
{
    if (s < 0 || s >= (long long)c.width * c.page.d) return false;
    const unsigned at = c.page.div((unsigned)s), slot = (unsigned)s - at * c.page.d;
    const int page = c.table[b * c.st + at];
    if (page < 0 || (unsigned)page >= c.pages) return false;
    *ok = page * c.sk[0] + slot * c.sk[1];
    *ov = page * c.sv[0] + slot * c.sv[1];
    return true;
}

struct AppendPlan {
    unsigned group;          // tokens of a CTA
    unsigned per_head;       // units of a head
    FastDiv by_head, by_unit, by_half, by_token;
    int across;              // the two pieces of a unit turn together (else neighbours within a piece)
};

struct TokenInfo {
    long long ok, ov;        // offsets in the caches, < 0: not written
    long long in[2], q, qo;  // offsets of the token in k, v, q, q_out
    int live, pos;
};

template <typename T, int N>
__global__ void __launch_bounds__(kThreads) k_append(AppendArgs a, AppendPlan p)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    TokenInfo *info = reinterpret_cast<TokenInfo *>(smem_raw);
    float2 *turn = reinterpret_cast<float2 *>(info + p.group);   // [group][rot / 2]
    const unsigned t = threadIdx.x, half = a.rot / 2;
    const unsigned total = a.batch * a.tokens;                   // below 2^31
    const unsigned first = blockIdx.x * p.group, n = min(p.group, total - first);
    pdl_wait();
    pdl_release();
    if (t < n) {
        const unsigned g = first + t, b = p.by_token.div(g), i = g - b * a.tokens;
        const int start = a.starts[b];
        int count = a.counts ? a.counts[b] : (int)a.tokens;
        bool bad = count < 0 || (unsigned)count > a.tokens || start < 0;
        TokenInfo x;
        x.live = (int)i < count;
        x.pos = a.positions ? a.positions[b * a.sp + i] : (int)((unsigned)start + i);
        x.ok = x.ov = -1;
        x.in[0] = b * a.si[0][0] + i * a.si[0][1];
        x.in[1] = b * a.si[1][0] + i * a.si[1][1];
        x.q = b * a.sq[0] + i * a.sq[1];
        x.qo = b * a.sqo[0] + i * a.sqo[1];
        long long ok = 0, ov = 0;
        if (x.live && start >= 0) {
            x.live = 1;
            if (place(a.c, b, (long long)start + i, &ok, &ov)) {
                x.ok = ok;
                x.ov = ov;
                x.live = 2;   // has a slot
            } else {
                bad = true;
            }
        }
        info[t] = x;
        if (bad && a.c.status) atomicOr(a.c.status, PER_DEVFLAG_BAD_INDEX);
    }
    __syncthreads();
    if (half) {
        for (unsigned u = t; u < n * half; u += kThreads) {
            const unsigned k = p.by_half.div(u), j = u - k * half;
            turn[u] = info[k].live ? cos_sin(a.inv_freq[j], info[k].pos) : make_float2(0.0f, 0.0f);
        }
        __syncthreads();
    }
    const unsigned heads = a.q_heads + 2 * a.c.heads, dim = a.c.dim;
    const unsigned rotated = p.across ? half / N : 0;            // units of a head that turn across their pieces
    const unsigned whole = heads * p.per_head;
    for (unsigned u = t; u < n * whole; u += kThreads) {
        const unsigned k = p.by_unit.div(u), r = u - k * whole;
        const unsigned h = p.by_head.div(r), w = r - h * p.per_head;
        const TokenInfo &x = info[k];
        const T *src;
        T *dst;
        bool turns_here = a.rot != 0, zero = false;
        if (h < a.q_heads) {
            src = static_cast<const T *>(a.q) + x.q + h * a.sq[2];
            dst = static_cast<T *>(a.q_out) + x.qo + h * a.sqo[2];
            zero = x.live == 0;
        } else {
            if (x.live < 2) continue;
            const unsigned hk = h - a.q_heads;
            if (hk < a.c.heads) {
                src = static_cast<const T *>(a.k) + x.in[0] + hk * a.si[0][2];
                dst = static_cast<T *>(a.c.k) + x.ok + hk * a.c.sk[2];
            } else {
                const unsigned hv = hk - a.c.heads;
                src = static_cast<const T *>(a.v) + x.in[1] + hv * a.si[1][2];
                dst = static_cast<T *>(a.c.v) + x.ov + hv * a.c.sv[2];
                turns_here = false;
            }
        }
        // the unit's two places
        unsigned p0, p1;
        bool across = false;
        if (turns_here && w < rotated) {
            across = true;
            if (N == 1 && a.interleaved) {
                p0 = 2 * w;
                p1 = p0 + 1;
            } else {
                p0 = w * N;
                p1 = p0 + half;
            }
        } else {
            p0 = turns_here ? 2 * rotated * N + (w - rotated) * 2 * N : w * 2 * N;
            p1 = p0 + N;
        }
        if (p0 >= dim) continue;
        const bool two = p1 < dim;
        Piece<T, N> y0, y1;
        if (zero) {
            y0.zero();
            y1.zero();
        } else {
            y0 = load_piece<T, N>(src + p0);
            if (two) y1 = load_piece<T, N>(src + p1);
            else y1.zero();
            const float2 *cs = turn + (size_t)k * half;
            if (across) {
                float f0[N], f1[N];
                y0.get(f0);
                y1.get(f1);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float2 z = cs[w * N + e];
                    const float g0 = f0[e] * z.x - f1[e] * z.y;
                    f1[e] = f1[e] * z.x + f0[e] * z.y;
                    f0[e] = g0;
                }
                y0.set(f0);
                y1.set(f1);
            } else if (N > 1 && turns_here && a.interleaved) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const unsigned at = s ? p1 : p0;
                    if (at >= a.rot) continue;
                    Piece<T, N> &y = s ? y1 : y0;
                    float f[N];
                    y.get(f);
#pragma unroll
                    for (int e = 0; e + 1 < N; e += 2) {
                        const float2 z = cs[(at + e) / 2];
                        const float g0 = f[e] * z.x - f[e + 1] * z.y;
                        f[e + 1] = f[e + 1] * z.x + f[e] * z.y;
                        f[e] = g0;
                    }
                    y.set(f);
                }
            }
        }
        store_piece<T, N>(dst + p0, y0);
        if (two) store_piece<T, N>(dst + p1, y1);
    }
}

template <typename T, int N>
cudaError_t launch_append_n(const AppendArgs &a, unsigned sms, cudaStream_t st)
{
    AppendPlan p{};
    const unsigned dim = a.c.dim, half = a.rot / 2, heads = a.q_heads + 2 * a.c.heads;
    p.across = a.rot && (N == 1 || !a.interleaved);
    const unsigned rotated = p.across ? half / N : 0;
    const unsigned copied = (dim + 2 * N - 1) / (2 * N);                              // units of a head without rotation
    p.per_head = std::max(copied, rotated + (dim - 2 * rotated * N + 2 * N - 1) / (2 * N));
    const unsigned whole = heads * p.per_head;                                        // at most 12288 x 129
    // about 8 units a thread, in no fewer CTAs than fill the SMs twice
    const unsigned total = a.batch * a.tokens;
    p.group = std::min(kMaxTokens, std::max(1u, 8 * kThreads / whole));
    while (p.group > 1 && (total + p.group - 1) / p.group < 2 * sms) p.group /= 2;
    p.by_head.set(p.per_head);
    p.by_unit.set(whole);
    p.by_half.set(std::max(half, 1u));
    p.by_token.set(a.tokens);
    const unsigned grid = (total + p.group - 1) / p.group;
    const size_t smem = p.group * (sizeof(TokenInfo) + half * sizeof(float2));
    return launch_clusters(k_append<T, N>, grid, kThreads, 1, smem, st, a, p);
}

// -- keep ---------------------------------------------------------------------------------------

constexpr int kAhead = 8;      // entries that a thread reads before it writes

struct Move {
    long long from[2], to[2];  // offsets in keys and values
};

template <typename T, int N>
__global__ void __launch_bounds__(kThreads) k_keep(KeepArgs a, unsigned splits, unsigned columns, FastDiv by_head)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Move *move = reinterpret_cast<Move *>(smem_raw);
    __shared__ unsigned ends;      // the first entry that is not moved
    const unsigned t = threadIdx.x, b = blockIdx.x / splits, part = blockIdx.x - b * splits;
    pdl_wait();
    pdl_release();
    int kept = a.kept[b];
    bool bad = kept < 0 || kept > (int)a.most;
    kept = min(max(kept, 0), (int)a.most);
    const long long start = a.lens[b];
    if (t == 0) ends = kept;
    __syncthreads();
    for (int j = t; j < kept; j += kThreads) {
        const int at = a.path[b * a.sp + j];
        const int before = j ? a.path[b * a.sp + j - 1] : -1;
        Move m;
        const bool fine = start >= 0 && at > before && at >= j && (unsigned)at < a.nodes &&
                          place(a.c, b, start + at, &m.from[0], &m.from[1]) &&
                          place(a.c, b, start + j, &m.to[0], &m.to[1]);
        if (fine) move[j] = m;
        else {
            atomicMin(&ends, (unsigned)j);
            bad = true;
        }
    }
    if (bad && a.c.status) atomicOr(a.c.status, PER_DEVFLAG_BAD_INDEX);
    __syncthreads();
    const int n = (int)ends;
    for (unsigned u = part * kThreads + t; u < columns; u += splits * kThreads) {
        const unsigned per = 2 * a.c.heads;               // heads of keys, then of values
        const unsigned h = by_head.div(u), w = u - h * by_head.d;
        const bool val = h >= a.c.heads;
        const unsigned hh = val ? h - a.c.heads : h;
        if (h >= per) continue;
        T *base = static_cast<T *>(val ? a.c.v : a.c.k) + hh * (val ? a.c.sv[2] : a.c.sk[2]) + w * N;
        for (int j0 = 0; j0 < n; j0 += kAhead) {
            Piece<T, N> y[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e)
                if (j0 + e < n) y[e] = load_piece<T, N>(base + move[j0 + e].from[val]);
#pragma unroll
            for (int e = 0; e < kAhead; ++e)
                if (j0 + e < n && move[j0 + e].from[val] != move[j0 + e].to[val])
                    store_piece<T, N>(base + move[j0 + e].to[val], y[e]);
        }
    }
}

template <typename T, int N>
cudaError_t launch_keep_n(const KeepArgs &a, unsigned sms, cudaStream_t st)
{
    const unsigned per_head = (a.c.dim + N - 1) / N, columns = 2 * a.c.heads * per_head;
    unsigned splits = 1;
    while (splits * kThreads < columns && a.batch * splits < 4 * sms) splits *= 2;
    FastDiv by_head;
    by_head.set(per_head);
    return launch_clusters(k_keep<T, N>, a.batch * splits, kThreads, 1, a.most * sizeof(Move), st, a, splits, columns, by_head);
}

template <typename T>
cudaError_t launch_append_t(const AppendArgs &a, unsigned sms, cudaStream_t st)
{
    return a.c.vec ? launch_append_n<T, Pack<T>::N>(a, sms, st) : launch_append_n<T, 1>(a, sms, st);
}

template <typename T>
cudaError_t launch_keep_t(const KeepArgs &a, unsigned sms, cudaStream_t st)
{
    return a.c.vec ? launch_keep_n<T, Pack<T>::N>(a, sms, st) : launch_keep_n<T, 1>(a, sms, st);
}

}  // namespace

cudaError_t launch_append(int type, const AppendArgs &a, cudaStream_t st)
{
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    const unsigned sms = (unsigned)dev.sms;
    if (type == PER_TYPE_F32) return launch_append_t<float>(a, sms, st);
    // 16-bit types differ in the rotation alone
    if (type == PER_TYPE_F16) return launch_append_t<__half>(a, sms, st);
    return launch_append_t<__nv_bfloat16>(a, sms, st);
}

cudaError_t launch_keep(int type, const KeepArgs &a, cudaStream_t st)
{
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    if (type == PER_TYPE_F32) return launch_keep_t<float>(a, (unsigned)dev.sms, st);
    return launch_keep_t<__nv_bfloat16>(a, (unsigned)dev.sms, st);   // 16 bits of either type move alike
}

}  // namespace gbper
