// k_scan.cu -- the gated linear recurrence h_t = w_t h_{t-1} + v_t over time, and its gradient.
//
// Mathematics.  A stretch of steps maps the state that comes in affinely: h -> A h + H, with A the
// product of its weights and H its end from a state of 0.  Two stretches join to (A1 A2, A2 H1 + H2), so
// a long sequence can be cut: every stretch is run once from 0 for its (A, H), the joints are
// scanned, and each stretch is run again from the state that really comes in, which needs no
// stored prefixes and rounds like the plain recurrence.  The gradient is the same recurrence in
// the other direction: with c_t = w_t g_t, g_t = gh_t + c_{t+1}, so c_t = w_t c_{t+1} + w_t gh_t.
// A weight of exactly 0 (a reset, a closed gate) drops what comes in whatever it holds, so it is a
// select, not a product; a product of weights that merely underflows is held at the smallest number,
// so that an infinite state is not dropped by it.  All of it is binary32.
//
// Work.  HBM bounds every case of some size (forward: two arrays read, one written; gradient: four or
// three read, two written).  A CTA takes a tile of CT channels and a stretch of steps; a thread takes VEC
// neighbouring channels (16 bytes) and R consecutive steps, so the rows of a tile are read in whole
// 128-byte lines; the threads' (A, H) are scanned by shuffles in a warp and by one thread a channel over the
// warps.  Where the channels alone do not fill the SMs, a cluster of up to 16 CTAs takes the same
// channels over consecutive stretches and exchanges the stretches' (A, H) through distributed shared
// memory, one hardware barrier a round.  The next rounds' rows arrive meanwhile: each thread
// copies what it will itself read (cp.async), so the copies need no barrier.
#include "ops_internal.cuh"

#include <algorithm>
#include <mutex>

namespace gbper {

namespace {

constexpr int kMaxCluster = 16;
constexpr int kMaxWarps = 8;
constexpr unsigned kFull = 0xffffffffu;

struct Gate {
    float w, v;   // the state's weight f and the input's 1 - f
};

// f = 1 / (1 + e), 1 - f = e f with e = exp(-a): neither loses digits to a subtraction.
template <bool SIG>
__device__ __forceinline__ Gate gate(float a)
{
    if (!SIG) return {a, 1.0f};
    const float e = ex2(a * -kLog2e);
    float f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(1.0f + e));
    return {f, f == 0.0f ? 1.0f : e * f};
}

// w h + more, a weight of 0 dropping whatever h holds
__device__ __forceinline__ float weigh(float w, float h, float more) { return w == 0.0f ? more : fmaf(w, h, more); }

// the product of two weights, 0 only if one of them is
__device__ __forceinline__ float chain(float a, float b)
{
    const float p = a * b;
    return p == 0.0f && a != 0.0f && b != 0.0f ? 1.4e-45f : p;
}

struct Stretch {
    float A, H;
};

__device__ __forceinline__ Stretch join(Stretch first, Stretch then)
{
    return {chain(first.A, then.A), weigh(then.A, first.H, then.H)};
}

// VEC values of T as they are in memory
template <int BYTES> struct Bits;
template <> struct Bits<16> { typedef uint4 type; };
template <> struct Bits<4> { typedef unsigned type; };
template <> struct Bits<2> { typedef unsigned short type; };

template <typename T, int VEC>
struct Cell {
    typedef typename Bits<VEC * (int)sizeof(T)>::type Raw;
    static __device__ __forceinline__ void unpack(const Raw &r, float *f)
    {
        if constexpr (VEC > 1) {
            Pack<T> p;
            p.raw = r;
            p.unpack(f);
        } else {
            T v;
            memcpy(&v, &r, sizeof(T));
            f[0] = to_f32(v);
        }
    }
    static __device__ __forceinline__ void store(T *at, const float *f)
    {
        if constexpr (VEC > 1) {
            Pack<T> p;
            p.pack(f);
            *reinterpret_cast<uint4 *>(at) = p.raw;
        } else {
            *at = from_f32<T>(f[0]);
        }
    }
};

template <int BYTES>
__device__ __forceinline__ void copy_async(void *smem, const void *global)
{
    const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(global) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s), "l"(global) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A thread's rows of NA arrays for the rounds ahead.  Values of 4 bytes and more are copied to a ring of
// ST rounds in shared memory, each thread reading only what it copied; single values of 2 bytes, which
// cp.async cannot copy, are held in registers one round ahead.
template <typename T, int VEC, int R, int NA, int ST>
struct Rows {
    typedef Cell<T, VEC> C;
    typedef typename C::Raw Raw;
    static constexpr int BYTES = VEC * (int)sizeof(T);
    static constexpr bool ASYNC = BYTES >= 4;
    static constexpr int AHEAD = ASYNC ? ST - 1 : 1;   // rounds requested before they are used
    Raw *ring;                      // [ST][NA][R][threads]
    Raw now[ASYNC ? 1 : NA][ASYNC ? 1 : R], next[ASYNC ? 1 : NA][ASYNC ? 1 : R];

    __device__ __forceinline__ Raw *slot(int round, int array, int i) const
    {
        return ring + (((round % ST) * NA + array) * R + i) * blockDim.x + threadIdx.x;
    }
    // requests rows [t0, t0 + R) of one array for `round`
    __device__ __forceinline__ void request(int round, int array, const T *p, long long stride, long long t0, long long steps, bool live)
    {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!live || t0 + i >= steps) continue;
            const Raw *from = reinterpret_cast<const Raw *>(p + (t0 + i) * stride);
            if constexpr (ASYNC) copy_async<BYTES>(slot(round, array, i), from);
            else next[array][i] = *from;
        }
    }
    __device__ __forceinline__ void requested() const
    {
        if constexpr (ASYNC) copies_commit();
    }
    // makes `round` readable
    __device__ __forceinline__ void arrive()
    {
        if constexpr (ASYNC) {
            copies_wait<ST - 2>();
        } else {
#pragma unroll
            for (int a = 0; a < NA; ++a)
#pragma unroll
                for (int i = 0; i < R; ++i) now[a][i] = next[a][i];
        }
    }
    __device__ __forceinline__ void read(int round, int array, int i, float *f) const
    {
        if constexpr (ASYNC) C::unpack(*slot(round, array, i), f);
        else C::unpack(now[array][i], f);
    }
};

// The scan of the threads' stretches over one round of a CTA (and its cluster).
template <int VEC, int LC>
struct Joints {
    static constexpr int CT = VEC * LC, RW = 32 / LC;
    Stretch *totals;   // [warps][CT]
    float *carry;      // [warps][CT] the state that comes into each warp's stretch
    float *state;      // [CT] the state that comes into the round
    Stretch *cluster;  // [2][csize][CT]
    unsigned csize, rank;

    static __host__ __device__ size_t bytes(int warps, unsigned csize)
    {
        return (size_t)CT * (warps * 12 + 4 + (csize > 1 ? 16 * csize : 0));
    }
    __device__ __forceinline__ Joints(unsigned char *mem, unsigned csize_, unsigned rank_) : csize(csize_), rank(rank_)
    {
        const int warps = blockDim.x >> 5;
        totals = reinterpret_cast<Stretch *>(mem);
        cluster = totals + warps * CT;
        carry = reinterpret_cast<float *>(cluster + (csize > 1 ? 2 * csize * CT : 0));
        state = carry + warps * CT;
    }
    // own: this thread's stretch, by channel; h receives the state that comes into it
    __device__ __forceinline__ void scan(int round, const Stretch *own, float *h)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lc = lane % LC, warps = blockDim.x >> 5;
        Stretch incl[VEC], excl[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            incl[e] = own[e];
            excl[e] = {1.0f, 0.0f};
        }
        if constexpr (RW > 1) {
#pragma unroll
            for (int o = LC; o < 32; o <<= 1)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const Stretch before{__shfl_up_sync(kFull, incl[e].A, o), __shfl_up_sync(kFull, incl[e].H, o)};
                    if (lane >= o) incl[e] = join(before, incl[e]);
                }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const Stretch before{__shfl_up_sync(kFull, incl[e].A, LC), __shfl_up_sync(kFull, incl[e].H, LC)};
                if (lane >= LC) excl[e] = before;
            }
        }
        if (lane >= 32 - LC) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) totals[warp * CT + lc * VEC + e] = incl[e];
        }
        __syncthreads();
        if (csize > 1) {
            Stretch *slot = cluster + (round & 1) * csize * CT;
            for (int ch = threadIdx.x; ch < CT; ch += blockDim.x) {
                Stretch all = totals[ch];
                for (int w = 1; w < warps; ++w) all = join(all, totals[w * CT + ch]);
                for (unsigned r = 0; r < csize; ++r) {
                    const unsigned to = cluster_smem_addr(slot + rank * CT + ch, r);
                    st_cluster_f32(to, all.A);
                    st_cluster_f32(to + 4, all.H);
                }
            }
            cluster_sync_all();
            for (int ch = threadIdx.x; ch < CT; ch += blockDim.x) {
                float c = state[ch], in = 0.0f;
                for (unsigned r = 0; r < csize; ++r) {
                    if (r == rank) in = c;
                    c = weigh(slot[r * CT + ch].A, c, slot[r * CT + ch].H);
                }
                state[ch] = c;
                for (int w = 0; w < warps; ++w) {
                    carry[w * CT + ch] = in;
                    in = weigh(totals[w * CT + ch].A, in, totals[w * CT + ch].H);
                }
            }
        } else {
            for (int ch = threadIdx.x; ch < CT; ch += blockDim.x) {
                float c = state[ch];
                for (int w = 0; w < warps; ++w) {
                    carry[w * CT + ch] = c;
                    c = weigh(totals[w * CT + ch].A, c, totals[w * CT + ch].H);
                }
                state[ch] = c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = weigh(excl[e].A, carry[warp * CT + lc * VEC + e], excl[e].H);
    }
};

// Where a CTA and a thread stand.
template <int VEC, int LC, int R>
struct Place {
    static constexpr int CT = VEC * LC, RW = 32 / LC;
    unsigned rank;
    long long b, tile, span, row0;   // sequence, steps a CTA takes a round, a cluster takes, this thread's first
    unsigned c0, ch;                 // the tile's first channel and this thread's
    int rounds;
    bool live;
    __device__ __forceinline__ Place(const ScanArgs &s, unsigned ctiles, unsigned csize)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        rank = blockIdx.x % csize;
        const unsigned id = blockIdx.x / csize;
        b = id / ctiles;
        c0 = id % ctiles * CT;
        ch = c0 + lane % LC * VEC;
        live = ch < s.channels;
        tile = (long long)(blockDim.x >> 5) * RW * R;
        span = tile * csize;
        row0 = rank * tile + (warp * RW + lane / LC) * R;
        rounds = (int)((s.steps + span - 1) / span);
    }
};

template <int R>
__device__ __forceinline__ unsigned reset_bits(const ScanArgs &s, long long b, long long t0)
{
    unsigned bits = 0;
    if (s.resets) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (t0 + i < s.steps && s.resets[b * s.sr[0] + (t0 + i) * s.sr[1]]) bits |= 1u << i;
    }
    return bits;
}

template <typename T, bool SIG, int VEC, int LC, int R, int ST>
__global__ void __launch_bounds__(kMaxWarps * 32) k_scan_fwd(ScanArgs s, unsigned ctiles, unsigned csize)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    typedef Rows<T, VEC, R, 2, ST> In;
    typedef Joints<VEC, LC> J;
    const Place<VEC, LC, R> me(s, ctiles, csize);
    In in;
    in.ring = reinterpret_cast<typename In::Raw *>(dyn);
    J joints(dyn + (In::ASYNC ? (size_t)ST * 2 * R * In::BYTES * blockDim.x : 0), csize, me.rank);
    pdl_wait();
    pdl_release();
    const T *a = static_cast<const T *>(s.a) + me.b * s.sa[0] + me.ch;
    const T *x = static_cast<const T *>(s.x) + me.b * s.sx[0] + me.ch;
    T *out = static_cast<T *>(s.out_h) + me.b * s.sh[0] + me.ch;
#pragma unroll
    for (int k = 0; k < In::AHEAD; ++k) {
        in.request(k, 0, a, s.sa[1], me.row0 + k * me.span, s.steps, me.live);
        in.request(k, 1, x, s.sx[1], me.row0 + k * me.span, s.steps, me.live);
        in.requested();
    }
    unsigned resets = reset_bits<R>(s, me.b, me.row0);
    for (unsigned ch = threadIdx.x; ch < (unsigned)J::CT; ch += blockDim.x)
        joints.state[ch] = s.h0 && me.c0 + ch < s.channels ? s.h0[me.b * s.channels + me.c0 + ch] : 0.0f;
    if (csize > 1) cluster_sync_all();   // every CTA of the cluster has started (and has read h0)
    for (int k = 0; k < me.rounds; ++k) {
        const long long t0 = me.row0 + k * me.span;
        in.arrive();
        float w[R][VEC], v[R][VEC];
        Stretch own[VEC];
        unsigned zero[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            own[e] = {1.0f, 0.0f};
            zero[e] = 0;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            in.read(k, 0, i, w[i]);
            in.read(k, 1, i, v[i]);
            const bool valid = me.live && t0 + i < s.steps, reset = resets >> i & 1u;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const Gate g = gate<SIG>(w[i][e]);
                if (SIG) v[i][e] = weigh(g.v, v[i][e], 0.0f);
                w[i][e] = reset ? 0.0f : g.w;
                if (!valid) {   // past the end: the state stays
                    w[i][e] = 1.0f;
                    v[i][e] = 0.0f;
                }
                zero[e] |= w[i][e] == 0.0f;
                own[e].H = weigh(w[i][e], own[e].H, v[i][e]);
                own[e].A *= w[i][e];
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (own[e].A == 0.0f && !zero[e]) own[e].A = 1.4e-45f;
        if (In::ASYNC || k + 1 < me.rounds) {
            const long long ahead = t0 + In::AHEAD * me.span;
            in.request(k + In::AHEAD, 0, a, s.sa[1], ahead, s.steps, me.live);
            in.request(k + In::AHEAD, 1, x, s.sx[1], ahead, s.steps, me.live);
            in.requested();
        }
        resets = reset_bits<R>(s, me.b, t0 + me.span);
        float h[VEC];
        joints.scan(k, own, h);
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[e] = weigh(w[i][e], h[e], v[i][e]);
            if (me.live && t0 + i < s.steps) Cell<T, VEC>::store(out + (t0 + i) * s.sh[1], h);
        }
    }
    if (s.last && me.rank == 0)
        for (unsigned ch = threadIdx.x; ch < (unsigned)J::CT && me.c0 + ch < s.channels; ch += blockDim.x)
            s.last[me.b * s.channels + me.c0 + ch] = joints.state[ch];
}

// The gradient, on arrays turned so that step 0 is the last one forward; s.h is shifted by one step, so
// that row t holds the state before that step (row steps - 1 is h0).
template <typename T, bool SIG, int VEC, int LC, int R, int ST>
__global__ void __launch_bounds__(kMaxWarps * 32) k_scan_bwd(ScanArgs s, unsigned ctiles, unsigned csize)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int NA = SIG ? 4 : 3;
    typedef Rows<T, VEC, R, NA, ST> In;
    typedef Joints<VEC, LC> J;
    const Place<VEC, LC, R> me(s, ctiles, csize);
    In in;
    in.ring = reinterpret_cast<typename In::Raw *>(dyn);
    J joints(dyn + (In::ASYNC ? (size_t)ST * NA * R * In::BYTES * blockDim.x : 0), csize, me.rank);
    pdl_wait();
    pdl_release();
    const T *a = static_cast<const T *>(s.a) + me.b * s.sa[0] + me.ch;
    const T *gh = static_cast<const T *>(s.gh) + me.b * s.sgh[0] + me.ch;
    const T *h = static_cast<const T *>(s.h) + me.b * s.sh[0] + me.ch;
    const T *x = SIG ? static_cast<const T *>(s.x) + me.b * s.sx[0] + me.ch : nullptr;
    T *ga = s.ga ? static_cast<T *>(s.ga) + me.b * s.sga[0] + me.ch : nullptr;
    T *gx = s.gx ? static_cast<T *>(s.gx) + me.b * s.sgx[0] + me.ch : nullptr;
    auto request = [&](int k, long long t0) {
        in.request(k, 0, a, s.sa[1], t0, s.steps, me.live);
        in.request(k, 1, gh, s.sgh[1], t0, s.steps, me.live);
        in.request(k, 2, h, s.sh[1], t0, s.steps - 1, me.live);
        if (SIG) in.request(k, 3, x, s.sx[1], t0, s.steps, me.live);
        in.requested();
    };
#pragma unroll
    for (int k = 0; k < In::AHEAD; ++k) request(k, me.row0 + k * me.span);
    unsigned resets = reset_bits<R>(s, me.b, me.row0);
    for (unsigned ch = threadIdx.x; ch < (unsigned)J::CT; ch += blockDim.x)
        joints.state[ch] = s.glast && me.c0 + ch < s.channels ? s.glast[me.b * s.channels + me.c0 + ch] : 0.0f;
    if (csize > 1) cluster_sync_all();
    for (int k = 0; k < me.rounds; ++k) {
        const long long t0 = me.row0 + k * me.span;
        in.arrive();
        if (!In::ASYNC && k + 1 < me.rounds) request(k + 1, t0 + me.span);
        const unsigned next_resets = reset_bits<R>(s, me.b, t0 + me.span);
        Stretch own[VEC];
        unsigned zero[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            own[e] = {1.0f, 0.0f};
            zero[e] = 0;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float w[VEC], g[VEC];
            in.read(k, 0, i, w);
            in.read(k, 1, i, g);
            const bool valid = me.live && t0 + i < s.steps, reset = resets >> i & 1u;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float f = reset ? 0.0f : gate<SIG>(w[e]).w;
                float in_c = weigh(f, g[e], 0.0f);
                if (!valid) {
                    f = 1.0f;
                    in_c = 0.0f;
                }
                zero[e] |= f == 0.0f;
                own[e].H = weigh(f, own[e].H, in_c);
                own[e].A *= f;
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (own[e].A == 0.0f && !zero[e]) own[e].A = 1.4e-45f;
        float c[VEC];
        joints.scan(k, own, c);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool valid = me.live && t0 + i < s.steps, reset = resets >> i & 1u;
            if (!valid) continue;
            float w[VEC], g[VEC], before[VEC], in_x[VEC], da[VEC], dx[VEC];
            in.read(k, 0, i, w);
            in.read(k, 1, i, g);
            in.read(k, 2, i, before);
            if (SIG) in.read(k, 3, i, in_x);
            if (t0 + i == s.steps - 1) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) before[e] = s.h0 ? s.h0[me.b * s.channels + me.ch + e] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const Gate f = gate<SIG>(w[e]);
                const float gt = g[e] + c[e];
                const float bt = reset ? 0.0f : before[e];
                if (SIG) {
                    const float slope = f.w * f.v;
                    da[e] = slope == 0.0f ? 0.0f : gt * (bt - in_x[e]) * slope;
                    dx[e] = weigh(f.v, gt, 0.0f);
                } else {
                    da[e] = reset ? 0.0f : gt * bt;
                    dx[e] = gt;
                }
                c[e] = weigh(reset ? 0.0f : f.w, gt, 0.0f);
            }
            if (ga) Cell<T, VEC>::store(ga + (t0 + i) * s.sga[1], da);
            if (gx) Cell<T, VEC>::store(gx + (t0 + i) * s.sgx[1], dx);
        }
        resets = next_resets;
        if (In::ASYNC) request(k + In::AHEAD, t0 + In::AHEAD * me.span);
    }
    if (s.gh0 && me.rank == 0)
        for (unsigned ch = threadIdx.x; ch < (unsigned)J::CT && me.c0 + ch < s.channels; ch += blockDim.x)
            s.gh0[me.b * s.channels + me.c0 + ch] = joints.state[ch];
}

// A few steps: one thread takes VEC channels through all of them.
template <typename T, bool SIG, int VEC>
__global__ void __launch_bounds__(128) k_scan_few(ScanArgs s)
{
    const unsigned per = s.channels / VEC;
    const unsigned id = blockIdx.x * 128 + threadIdx.x;
    pdl_wait();
    pdl_release();
    if (id >= per * s.batch) return;
    const long long b = id / per;
    const unsigned ch = id % per * VEC;
    const T *a = static_cast<const T *>(s.a) + b * s.sa[0] + ch;
    const T *x = static_cast<const T *>(s.x) + b * s.sx[0] + ch;
    T *out = static_cast<T *>(s.out_h) + b * s.sh[0] + ch;
    typedef typename Cell<T, VEC>::Raw Raw;
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = s.h0 ? s.h0[b * s.channels + ch + e] : 0.0f;
    for (long long t = 0; t < s.steps; ++t) {
        float w[VEC], v[VEC];
        const Raw ra = *reinterpret_cast<const Raw *>(a + t * s.sa[1]), rx = *reinterpret_cast<const Raw *>(x + t * s.sx[1]);
        const bool reset = s.resets && s.resets[b * s.sr[0] + t * s.sr[1]];
        Cell<T, VEC>::unpack(ra, w);
        Cell<T, VEC>::unpack(rx, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const Gate g = gate<SIG>(w[e]);
            h[e] = weigh(reset ? 0.0f : g.w, h[e], SIG ? weigh(g.v, v[e], 0.0f) : v[e]);
        }
        Cell<T, VEC>::store(out + t * s.sh[1], h);
    }
    if (s.last) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) s.last[b * s.channels + ch + e] = h[e];
    }
}

// ---- launches --------------------------------------------------------------------------------

#ifndef FST
#define FST 3
#endif
#ifndef BST
#define BST 3
#endif
#ifndef FR16
#define FR16 4
#endif
#ifndef BR16
#define BR16 2
#endif
#ifndef FR32
#define FR32 4
#endif
#ifndef BR32
#define BR32 2
#endif
#ifndef FILL
#define FILL 2
#endif
#ifndef MAXCL
#define MAXCL 16
#endif

// The tiles: 16 bytes a thread where the arrays allow it, else one value.
template <typename T, bool WIDE>
struct Tile;
template <> struct Tile<float, true> { static constexpr int VEC = 4, LC = 8, FR = FR32, BR = BR32; };
template <> struct Tile<__half, true> { static constexpr int VEC = 8, LC = 8, FR = FR16, BR = BR16; };
template <> struct Tile<__nv_bfloat16, true> { static constexpr int VEC = 8, LC = 8, FR = FR16, BR = BR16; };
template <> struct Tile<float, false> { static constexpr int VEC = 1, LC = 32, FR = 16, BR = 8; };
template <> struct Tile<__half, false> { static constexpr int VEC = 1, LC = 32, FR = 16, BR = 8; };
template <> struct Tile<__nv_bfloat16, false> { static constexpr int VEC = 1, LC = 32, FR = 16, BR = 8; };

template <typename K>
cudaError_t allow(K kernel, int smem)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

template <typename T, bool SIG, bool WIDE, bool BACK>
cudaError_t launch_tiles(const ScanArgs &a, const DeviceInfo &dev, cudaStream_t st)
{
    typedef Tile<T, WIDE> S;
    constexpr int R = BACK ? S::BR : S::FR, NA = BACK ? (SIG ? 4 : 3) : 2, ST = BACK ? BST : FST;
    constexpr int BYTES = S::VEC * (int)sizeof(T), CT = S::VEC * S::LC, RW = 32 / S::LC;
    auto kernel = [] {
        if constexpr (BACK) return k_scan_bwd<T, SIG, S::VEC, S::LC, R, ST>;
        else return k_scan_fwd<T, SIG, S::VEC, S::LC, R, ST>;
    }();
    auto smem_of = [](int warps, unsigned csize) {
        return (BYTES >= 4 ? (size_t)ST * NA * R * BYTES * warps * 32 : 0) + Joints<S::VEC, S::LC>::bytes(warps, csize);
    };
    {
        static std::mutex mu;
        static bool done[64] = {};
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev.device]) {
            const cudaError_t e = allow(kernel, (int)smem_of(kMaxWarps, kMaxCluster));
            if (e != cudaSuccess) return e;
            done[dev.device] = true;
        }
    }
    const unsigned ctiles = (a.channels + CT - 1) / CT;
    const unsigned long long tiles = (unsigned long long)ctiles * a.batch;
    // warps: no more than the steps need; then CTAs over time until the SMs are filled, as long as each
    // has a stretch of its own
    int warps = 1;
    while (warps < kMaxWarps && (long long)warps * RW * R < a.steps) warps *= 2;
    unsigned csize = 1;
    while (csize < MAXCL && tiles * csize < (unsigned)FILL * dev.sms && (long long)warps * RW * R * csize < a.steps) csize *= 2;
    if (tiles * csize > 0x7fffffffull) return cudaErrorInvalidConfiguration;
    return launch_clusters(kernel, (unsigned)(tiles * csize), warps * 32, csize, smem_of(warps, csize), st, a, ctiles, csize);
}

bool aligned16(const void *p, const long long st[2], const ScanArgs &a, unsigned e)
{
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.batch <= 1 || st[0] * (long long)e % 16 == 0) &&
                  (a.steps <= 1 || st[1] * (long long)e % 16 == 0));
}

template <typename T, bool SIG>
cudaError_t fwd_t(const ScanArgs &a, const DeviceInfo &dev, cudaStream_t st)
{
    constexpr unsigned e = sizeof(T), P = 16 / e;
    const bool wide = a.channels % P == 0 && aligned16(a.a, a.sa, a, e) && aligned16(a.x, a.sx, a, e) &&
                      aligned16(a.out_h, a.sh, a, e);
    if (a.steps <= 4) {
        const unsigned long long threads = (unsigned long long)a.channels / (wide ? P : 1) * a.batch;
        const unsigned grid = (unsigned)((threads + 127) / 128);
        if (wide) return launch_clusters(k_scan_few<T, SIG, (int)P>, grid, 128, 1, 0, st, a);
        return launch_clusters(k_scan_few<T, SIG, 1>, grid, 128, 1, 0, st, a);
    }
    return wide ? launch_tiles<T, SIG, true, false>(a, dev, st) : launch_tiles<T, SIG, false, false>(a, dev, st);
}

template <typename T, bool SIG>
cudaError_t bwd_t(const ScanArgs &a, const DeviceInfo &dev, cudaStream_t st)
{
    constexpr unsigned e = sizeof(T), P = 16 / e;
    const bool wide = a.channels % P == 0 && aligned16(a.a, a.sa, a, e) && aligned16(a.x, a.sx, a, e) &&
                      aligned16(a.h, a.sh, a, e) && aligned16(a.gh, a.sgh, a, e) && aligned16(a.ga, a.sga, a, e) &&
                      aligned16(a.gx, a.sgx, a, e);
    return wide ? launch_tiles<T, SIG, true, true>(a, dev, st) : launch_tiles<T, SIG, false, true>(a, dev, st);
}

// What a pass of no steps leaves: the state that came in.
cudaError_t copy_state(float *to, const float *from, const ScanArgs &a, cudaStream_t st)
{
    if (!to || to == from) return cudaSuccess;
    const size_t bytes = (size_t)a.batch * a.channels * sizeof(float);
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, bytes, st);
}

void turn(const void **p, long long st[2], const ScanArgs &a, unsigned e, long long shift)
{
    if (*p) *p = static_cast<const char *>(*p) + (a.steps - 1 - shift) * st[1] * (long long)e;
    st[1] = -st[1];
}

}  // namespace

cudaError_t launch_scan_forward(int type, bool sigmoid, const ScanArgs &a, cudaStream_t st)
{
    if (a.steps == 0) return copy_state(a.last, a.h0, a, st);
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    if (type == PER_TYPE_F32) return sigmoid ? fwd_t<float, true>(a, dev, st) : fwd_t<float, false>(a, dev, st);
    if (type == PER_TYPE_F16) return sigmoid ? fwd_t<__half, true>(a, dev, st) : fwd_t<__half, false>(a, dev, st);
    return sigmoid ? fwd_t<__nv_bfloat16, true>(a, dev, st) : fwd_t<__nv_bfloat16, false>(a, dev, st);
}

cudaError_t launch_scan_backward(int type, bool sigmoid, const ScanArgs &args, cudaStream_t st)
{
    ScanArgs a = args;
    if (a.steps == 0) return copy_state(a.gh0, a.glast, a, st);
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    const unsigned bytes = type == PER_TYPE_F32 ? 4 : 2;
    turn(&a.a, a.sa, a, bytes, 0);
    turn(&a.x, a.sx, a, bytes, 0);
    turn(&a.gh, a.sgh, a, bytes, 0);
    turn(&a.h, a.sh, a, bytes, 1);
    turn(const_cast<const void **>(&a.ga), a.sga, a, bytes, 0);
    turn(const_cast<const void **>(&a.gx), a.sgx, a, bytes, 0);
    const void *r = a.resets;
    turn(&r, a.sr, a, 1, 0);
    a.resets = static_cast<const uint8_t *>(r);
    if (type == PER_TYPE_F32) return sigmoid ? bwd_t<float, true>(a, dev, st) : bwd_t<float, false>(a, dev, st);
    if (type == PER_TYPE_F16) return sigmoid ? bwd_t<__half, true>(a, dev, st) : bwd_t<__half, false>(a, dev, st);
    return sigmoid ? bwd_t<__nv_bfloat16, true>(a, dev, st) : bwd_t<__nv_bfloat16, false>(a, dev, st);
}

}  // namespace gbper
