// k_scan.cu -- the gated linear recurrence h_t = w_t h_{t-1} + v_t over time, and its gradient.
//
// Mathematics.  A stretch of steps maps the state that comes in affinely: h -> A h + H, with A the
// product of its weights and H its end from a state of 0.  Two stretches join to (A1 A2, A2 H1 + H2), so
// a long sequence can be cut: every stretch is run once from 0 for its (A, H), the joints are
// scanned, and each stretch is run again from the state that really comes in, which needs no
// stored prefixes and rounds like the plain recurrence.  The gradient is the same recurrence in
// the other direction: with c_t = w_t g_t, g_t = gh_t + c_{t+1}, so c_t = w_t (gh_t + c_{t+1}).
// A weight of exactly 0 (a reset, a closed gate) drops what comes in whatever it holds, so it is a
// select, not a product; a product of weights that merely underflows is held at the smallest number,
// so that an infinite state is not dropped by it.  All of it is binary32.
//
// Work.  HBM bounds every case of some size (forward: two arrays read, one written; gradient: four or
// three read, two written).  A warp takes a strip of 16 channels and works through time in tiles of 4 x N
// steps: its lanes copy the tile's rows 16 bytes a copy (cp.async) some tiles ahead into a ring in shared
// memory, and read it the other way round: a lane takes two neighbouring channels and N consecutive
// steps, sweeps them once from 0 for its (A, H) and, when the state that comes in is known, once more for
// the outputs, so only the joints of four groups of lanes are left to be scanned by shuffles.  Where there
// are strips enough, nothing else is needed: no barrier.  Else several warps of a CTA take consecutive tiles
// of a strip (one CTA barrier a round), and then a cluster of up to 16 CTAs: each CTA sends its round's
// (A, H) to the others by asynchronous stores into their shared memory, which count down a barrier there
// (no fence, so output stores in flight are not waited for), and only then finishes the round before:
// the exchange runs beside the next round's first sweep.  (A remote store takes about 8 cycles of the
// receiver: with one warp's stretch a message, 16 CTAs to 16, the exchange took 3.6 us a round.)  Where the
// channels are many, or the steps few, one thread a channel (k_scan_few) takes fewer instructions.
//
// Measured (GB300): 64 x 1024 x 1024 f32 forward 121 us, 6.7 TB/s; both passes of 8 x 16384 x 1024 f32 742 us, 5.8 TB/s;
// 16 x 2048 x 2048 bf16 sigmoid gradient 176 us, 4.6 TB/s (its instructions bound it); one sequence of 65537 x
// 1024 bf16 149 us, 2.7 TB/s (the joints); one step of 64 x 2048 2.0 us.
#include "ops_internal.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>

namespace gbper {

namespace {

// Measured on 64 x 1024 x 1024 bf16 with sigmoid gates, forward and gradient, and on one sequence of 65537 x 1024 (a
// cluster), us.  Steps of a lane in a tile: 8 82 and 170, 16 86 and 198 (registers); with a cluster, where the
// joints are the larger part, 16 141, 8 149.  Tiles in a ring: 2 82 and 170, 3 82 and 172; with a cluster 3 (two
// under way, one arriving) 141, 4 165.
constexpr int kLaneSteps = 8, kLaneStepsCluster16 = 16;
constexpr int kRing = 2, kRingCluster = 3;
constexpr int kCtasPerSm = 4;   // what registers are kept for (CTAs of 4 warps): 4 82, 170, 141; 3 83, 188, 162; 5 89, 203, 147
// With a cluster the gradient's ring takes 78 to 111 KB a CTA, so that two fit and may have twice the registers (one sequence
// of 65537 x 1023 binary32 with sigmoid gates 710 us, with those of four 804).
constexpr int kCtasPerSmBack = 2;

constexpr int kMaxCluster = 16;
constexpr int kWarps = 4;     // of a CTA at most: strips side by side, times tiles one after the other
constexpr int kStrip = 16;    // channels of a warp
constexpr int kGroups = 4;    // groups of 8 lanes, one after the other in time
constexpr float kInf = __builtin_huge_valf();
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Gate {
    float w, v;   // the state's weight f and the input's 1 - f
};

// exp(-a) of two gates, by powers of 2.  x = -a log2(e) is off by its rounding, a relative |a| 2^-24 of the power and
// 2^-22 more of its own (4e-6 at a gate of 80).  For binary32 gates that is made up for: 2^x times 1 - (a + x ln 2), the
// difference small and good to 2^-24 of itself by two fused steps over ln 2 in two parts.  (Not finite below
// about -88, where it would be 0 or NaN as a weight and the careful way is taken.)  The 16-bit passes, which
// their instructions bound and whose gates are rounded to 2^-9 or 2^-12 themselves, take 2^x.
template <typename T>
__device__ __forceinline__ F2 exp_minus(F2 a)
{
    const F2 x = a * F2{-kLog2e, -kLog2e};
    F2 e{ex2(x.x), ex2(x.y)};
    if constexpr (sizeof(T) == 4) {
        constexpr float kLn2 = 0.693147182f, kLn2Rest = -1.90465421e-9f;
        const F2 minus{-1.0f, -1.0f};
        const F2 r = fma2(x, F2{-kLn2Rest, -kLn2Rest}, fma2(x, F2{-kLn2, -kLn2}, a * minus));
        e = fma2(e, r, e);
    }
    return e;
}

// e f, at most 1 as 1 - f is.  (Its roundings can take it to 1 + 2^-23, and binary32's lowest value times that, a mask,
// would be infinite; those of 16-bit types are far enough from there.)  NaN gives 0.
__device__ __forceinline__ float at_most_1(float e, float f)
{
    float v;
    asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(v) : "f"(e), "f"(f));
    return v;
}

// f = 1 / (1 + e), 1 - f = e f with e = exp(-a): neither loses digits to a subtraction.  (f below 2^-126 is 0.)
template <typename T, bool SIG>
__device__ __forceinline__ Gate gate(float a)
{
    if (!SIG) return {a, 1.0f};
    const float e = sizeof(T) == 4 ? expf(-a) : ex2(a * -kLog2e), f = rcp(1.0f + e);
    const float v = f == 0.0f ? 1.0f : e * f;
    return {f, sizeof(T) == 4 && v > 1.0f ? 1.0f : v};
}

// the same of two gates that are not 0
template <typename T>
__device__ __forceinline__ void gates(F2 a, F2 &w, F2 &v)
{
    const F2 e = exp_minus<T>(a);
    const F2 d = e + F2{1.0f, 1.0f};
    w = {rcp(d.x), rcp(d.y)};
    if constexpr (sizeof(T) == 4) v = {at_most_1(e.x, w.x), at_most_1(e.y, w.y)};
    else v = e * w;
}

// w h + more, a weight of 0 dropping whatever h holds
__device__ __forceinline__ float weigh(float w, float h, float more) { return w == 0.0f ? more : fmaf(w, h, more); }

// A stretch of steps.  A is NaN where the stretch drops what comes in (a weight of exactly 0 in it), and is
// never 0: a product that underflows is held at the smallest number of its sign, so that an infinite state times
// it stays infinite.  (A weight of NaN makes H NaN too.)
struct Stretch {
    float A, H;
};

// (by its bits: copysignf takes the long sequence to 162 us, this to 151)
__device__ __forceinline__ float nonzero(float a)
{
    int bits = __float_as_int(a);
    if (a == 0.0f) bits |= 1;
    return __int_as_float(bits);
}

__device__ __forceinline__ float apply(Stretch s, float h)
{
    const float r = fmaf(s.A, h, s.H);
    return s.A == s.A ? r : s.H;
}

__device__ __forceinline__ Stretch join(Stretch first, Stretch then)
{
    return {nonzero(first.A * then.A), apply(then, first.H)};
}

__device__ __forceinline__ Stretch shfl_up(Stretch s, int o)
{
    return {__shfl_up_sync(kFull, s.A, o), __shfl_up_sync(kFull, s.H, o)};
}
__device__ __forceinline__ Stretch shfl(Stretch s, int lane)
{
    return {__shfl_sync(kFull, s.A, lane), __shfl_sync(kFull, s.H, lane)};
}

// ---- the ring ------------------------------------------------------------------------------

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

template <typename T>
__device__ __forceinline__ F2 unpack2(const T *p);
template <> __device__ __forceinline__ F2 unpack2<float>(const float *p)
{
    const float2 v = *reinterpret_cast<const float2 *>(p);
    return {v.x, v.y};
}
template <> __device__ __forceinline__ F2 unpack2<__nv_bfloat16>(const __nv_bfloat16 *p)
{
    const unsigned w = *reinterpret_cast<const unsigned *>(p);
    return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
}
template <> __device__ __forceinline__ F2 unpack2<__half>(const __half *p)
{
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(p));
    return {v.x, v.y};
}

// stores a lane's two channels; WIDE: both exist and lie on a boundary of the pair
template <typename T, bool WIDE>
__device__ __forceinline__ void store2(T *p, F2 v, bool second)
{
    if constexpr (!WIDE) {
        p[0] = from_f32<T>(v.x);
        if (second) p[1] = from_f32<T>(v.y);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float2 *>(p) = make_float2(v.x, v.y);
    } else if constexpr (std::is_same<T, __half>::value) {
        *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(v.x, v.y);
    } else {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
    }
}

// A warp's tiles of NA arrays in shared memory, ST of them.  A group's 16 rows lie together, with a pad
// between groups that puts the four groups of a read into different banks.
template <typename T, int N, int NA, int ST, bool WIDE>
struct Ring {
    static constexpr int ROW = kStrip * (int)sizeof(T);
    static constexpr int GROUP = N * ROW + ROW;
    static constexpr int SLOT = kGroups * GROUP;
    static constexpr int BYTES = ST * NA * SLOT;       // of a warp
    unsigned char *mem;

    __device__ __forceinline__ unsigned char *slot(int tile, int array) const { return mem + (tile % ST * NA + array) * SLOT; }

    // requests rows [t0, t0 + (kGroups * N)) of an array, of which those below `steps` exist; p: the strip's first
    // channel, of which `channels` exist
    __device__ __forceinline__ void request(int tile, int array, const T *p, long long stride, long long t0, long long steps, int channels) const
    {
        const int lane = threadIdx.x & 31;
        unsigned char *to = slot(tile, array);
        constexpr int PIECE = WIDE ? 16 : (int)sizeof(T), PER = ROW / PIECE, ROWS = 32 / PER;
        const int c = lane % PER * (PIECE / (int)sizeof(T)), r0 = lane / PER;
        if (c >= channels) return;
        const long long left = steps - t0 - r0;
        const T *from = p + c + (t0 + r0) * stride;
        auto copy = [&](int i) {
            const int r = i * ROWS + r0;
            unsigned char *at = to + r / N * GROUP + r % N * ROW + lane % PER * PIECE;
            const T *src = from + i * (long long)ROWS * stride;
            if constexpr (PIECE >= 4) copy_async<PIECE>(at, src);
            else *reinterpret_cast<T *>(at) = *src;   // too small for an asynchronous copy
        };
        if (t0 + kGroups * N <= steps) {
#pragma unroll
            for (int i = 0; i < (kGroups * N) / ROWS; ++i) copy(i);
        } else {
#pragma unroll
            for (int i = 0; i < (kGroups * N) / ROWS; ++i)
                if (i * ROWS < left) copy(i);
        }
    }
    // this lane's two channels of its step i
    __device__ __forceinline__ F2 read(int tile, int array, int i) const
    {
        const int lane = threadIdx.x & 31;
        return unpack2<T>(reinterpret_cast<const T *>(slot(tile, array) + (lane / 8 * GROUP + lane % 8 * 2 * (int)sizeof(T)) + i * ROW));
    }
};

// ---- the partners of a cluster ------------------------------------------------------------

__device__ __forceinline__ unsigned smem_u32(const void *p) { return (unsigned)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(unsigned bar)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(unsigned bar, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// What the phase counted was stored by other CTAs of the cluster, so the acquire is at its scope (the default is the
// CTA's).
__device__ __forceinline__ bool mbar_try(unsigned bar, unsigned parity)
{
    unsigned ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Waits for the phase of the given parity to end; false when it has not after `limit` ms.
__device__ __noinline__ bool mbar_wait_long(unsigned bar, unsigned parity, unsigned limit)
{
    unsigned long long began, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(began));
    for (int tries = 0; tries < 1 << 24; ++tries) {
        if (mbar_try(bar, parity)) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (now - began > limit * 1000000ull) return false;
    }
    return false;
}
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned parity, unsigned limit)
{
    return mbar_try(bar, parity) || mbar_wait_long(bar, parity, limit);
}
__device__ __forceinline__ void store_async(unsigned to, uint4 v, unsigned bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar) : "memory");
}
__device__ __forceinline__ unsigned in_cta(unsigned addr, unsigned rank)
{
    unsigned r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// Rounds whose joints have places of their own.  A CTA sends round k + 4 after finishing round k + 2, so
// after this CTA sent round k + 2, so after this CTA finished round k: nothing is overwritten unread.  A warp that
// sends and has given up a wait does not know that, so it sends nothing more; the other CTAs then give up too.
constexpr int kDepth = 4;

__device__ __forceinline__ uint4 packed(const Stretch (&s)[2])
{
    return make_uint4(__float_as_uint(s[0].A), __float_as_uint(s[0].H), __float_as_uint(s[1].A), __float_as_uint(s[1].H));
}
__device__ __forceinline__ void unpacked(uint4 v, Stretch (&s)[2])
{
    s[0] = {__uint_as_float(v.x), __uint_as_float(v.y)};
    s[1] = {__uint_as_float(v.z), __uint_as_float(v.w)};
}

// A strip's tiles, joined over a warp's groups, the CTA's warps (`times` tiles of one strip one after the
// other), its cluster and the rounds.
template <bool CLUSTER>
struct Joints {
    uint4 *tiles;               // [kDepth][times][8] of the strip: two channels' (A, H) of each tile
    uint4 *slots;               // [kDepth][csize][8] of the strip: of each CTA
    unsigned long long *bar;    // [kDepth] of the strip
    unsigned csize, rank;
    int times, time;            // tiles of a strip in a round of the CTA, and which is this warp's
    F2 state;                   // what comes into the round, alike in all groups and warps of the strip
    bool lost = false, sends;   // sends: this warp tells the other CTAs of the stretches

    static __host__ __device__ size_t bytes(int times, unsigned csize)   // of a strip
    {
        return (times > 1 || CLUSTER ? kDepth * 128 * (size_t)times : 0) + (CLUSTER ? kDepth * (8 + 128 * (size_t)csize) : 0);
    }

    // mem: strips x bytes(times, csize); the whole cluster calls
    __device__ __forceinline__ void begin(const ScanArgs &args, unsigned char *mem, int strip, int times_, int time_, unsigned csize_, unsigned rank_)
    {
        csize = csize_;
        rank = rank_;
        times = times_;
        time = time_;
        tiles = reinterpret_cast<uint4 *>(mem + strip * bytes(times, csize));
        if (!CLUSTER) return;
        sends = time == times - 1 && rank + 1 != args.withhold;
        slots = tiles + kDepth * times * 8;
        bar = reinterpret_cast<unsigned long long *>(slots + kDepth * csize * 8);
        if (time == 0 && (threadIdx.x & 31) == 0) {
            for (int i = 0; i < kDepth; ++i) mbar_init(smem_u32(&bar[i]));
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            for (int i = 0; i < kDepth; ++i) mbar_expect(smem_u32(&bar[i]), csize * 128);
        }
        cluster_sync_all();   // every CTA's barriers are ready (and every CTA has read the first state)
    }

    // A, H: this lane's stretch where it is plain (A not 0, H finite; `resets` drops what comes in), else `own`.
    // Leaves the stretch of the groups before in `before` and that of the warp in `all`, and makes it known.
    __device__ __forceinline__ void first(int round, bool plain, F2 A, F2 H, bool resets, const Stretch (&own)[2],
                                          Stretch (&before)[2], Stretch (&all)[2])
    {
        const int lane = threadIdx.x & 31;
        if (__all_sync(kFull, plain)) {
            // Every lane's own numbers are finite, but what they join to need not be: a stretch that drops what
            // comes in leaves it out, which a product with 0 would not do to an infinite sum; which stretches drop
            // is told by the resets.
            const unsigned drops = __ballot_sync(kFull, resets);
#pragma unroll
            for (int o = 8; o < 32; o <<= 1) {
                const F2 a{__shfl_up_sync(kFull, A.x, o), __shfl_up_sync(kFull, A.y, o)};
                const F2 h{__shfl_up_sync(kFull, H.x, o), __shfl_up_sync(kFull, H.y, o)};
                // the groups that this lane's stretch takes in by now: its own, then the one before too
                const unsigned own_groups = o == 8 ? 0xffu << (lane & 24) : (0xffu << (lane & 24)) | (0xffu << (lane & 24)) >> 8;
                if (lane >= o && !(drops & own_groups)) {
                    H = fma2(A, h, H);
                    A = A * a;
                    if (o == 8) A = {nonzero(A.x), nonzero(A.y)};   // (it may meet an infinite sum)
                }
            }
            const bool earlier = (drops & ((1u << (lane & 24)) - 1u)) != 0u;
            const float nan = __int_as_float(0x7fffffff);
            const F2 ba{__shfl_up_sync(kFull, A.x, 8), __shfl_up_sync(kFull, A.y, 8)};
            before[0] = {earlier ? nan : nonzero(ba.x), __shfl_up_sync(kFull, H.x, 8)};
            before[1] = {earlier ? nan : nonzero(ba.y), __shfl_up_sync(kFull, H.y, 8)};
            const int end = 24 + lane % 8;
            const F2 aa{__shfl_sync(kFull, A.x, end), __shfl_sync(kFull, A.y, end)};
            all[0] = {drops ? nan : nonzero(aa.x), __shfl_sync(kFull, H.x, end)};
            all[1] = {drops ? nan : nonzero(aa.y), __shfl_sync(kFull, H.y, end)};
        } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                Stretch incl = own[c];
#pragma unroll
                for (int o = 8; o < 32; o <<= 1) {
                    const Stretch b = shfl_up(incl, o);
                    if (lane >= o) incl = join(b, incl);
                }
                const Stretch b = shfl_up(incl, 8), e = shfl(incl, 24 + lane % 8);
                before[c] = b;
                all[c] = e;
            }
        }
        if (times == 1 && !CLUSTER) return;
        const unsigned place = round % kDepth;
        uint4 *mine = tiles + place * times * 8 + lane % 8;
        if (lane < 8) mine[time * 8] = packed(all);
        __syncthreads();
        if (CLUSTER && sends) {   // the CTA's stretch, to four CTAs at a time
            Stretch sum[2], next[2];
            unpacked(mine[0], sum);
            for (int i = 1; i < times; ++i) {
                unpacked(mine[i * 8], next);
                sum[0] = join(sum[0], next[0]);
                sum[1] = join(sum[1], next[1]);
            }
            const unsigned to = smem_u32(slots + (place * csize + rank) * 8 + lane % 8), b = smem_u32(&bar[place]);
            for (unsigned r = lane / 8; r < csize; r += 4) store_async(in_cta(to, r), packed(sum), in_cta(b, r));
        }
    }

    // the state that comes into this lane's steps; moves `state` on
    __device__ __forceinline__ F2 second(const ScanArgs &args, int round, const Stretch (&before)[2], const Stretch (&all)[2])
    {
        const int lane = threadIdx.x & 31;
        F2 in = state;
        if (times == 1 && !CLUSTER) {
            state = {apply(all[0], in.x), apply(all[1], in.y)};
        } else {
            const unsigned place = round % kDepth;
            if (CLUSTER) {
                const unsigned b = smem_u32(&bar[place]);
                if (!lost) lost = !mbar_wait(b, round / kDepth & 1, args.wait_ms);
                if (__any_sync(kFull, lost)) {   // the status and the states say so
                    lost = true;
                    sends = false;
                    in = state = {__int_as_float(0x7fffffff), __int_as_float(0x7fffffff)};
                } else {
                    if (lane == 0 && time == 0) mbar_expect(b, csize * 128);   // for the round that uses it next
                    const uint4 *from = slots + place * csize * 8 + lane % 8;
                    F2 s = state;
#pragma unroll 4
                    for (unsigned r = 0; r < csize; ++r) {
                        if (r == rank) in = s;
                        Stretch next[2];
                        unpacked(from[r * 8], next);
                        s = {apply(next[0], s.x), apply(next[1], s.y)};
                    }
                    state = s;
                }
            }
            F2 s = in;
            const uint4 *mine = tiles + place * times * 8 + lane % 8;
            for (int i = 0; i < times; ++i) {
                if (i == time) in = s;
                Stretch next[2];
                unpacked(mine[i * 8], next);
                s = {apply(next[0], s.x), apply(next[1], s.y)};
            }
            if (!CLUSTER) state = s;
        }
        return lane >= 8 ? F2{apply(before[0], in.x), apply(before[1], in.y)} : in;
    }

    // nothing of this CTA is read or written any more when the whole cluster has finished every round
    __device__ __forceinline__ void end(const ScanArgs &args) const
    {
        if (!CLUSTER) return;
        cluster_sync_all();
        if (lost) {
            if (args.status && (threadIdx.x & 31) == 0) atomicOr(args.status, PER_DEVFLAG_TIMEOUT);
            // what the others sent and this CTA did not wait for is on its way at most: its memory stays until
            // that has arrived
            for (int i = 0; i < 20; ++i) __nanosleep(50000);
        }
    }
};

// Where a warp and a lane stand.
template <int N>   // steps of a lane in a tile
struct Place {
    unsigned rank;
    int strip, time;         // which of the CTA's strips, which of its tiles
    int c0, channels, ch;    // the strip's first channel, how many of its channels exist, this lane's first
    long long b, span, t0;   // sequence, steps a cluster takes a round, this warp's first step
    int rounds, off;         // off: this lane's first step in a tile
    bool live, second;       // this lane's first and second channel exist
    __device__ __forceinline__ Place(const ScanArgs &s, unsigned ctiles, unsigned csize, int times)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, strips = (int)(blockDim.x >> 5) / times;
        strip = warp % strips;
        time = warp / strips;
        rank = blockIdx.x % csize;
        const unsigned id = blockIdx.x / csize;
        b = id / ctiles;
        c0 = (int)(id % ctiles * strips + strip) * kStrip;
        channels = max(0, min(kStrip, (int)s.channels - c0));
        ch = c0 + lane % 8 * 2;
        live = ch < (int)s.channels;
        second = ch + 1 < (int)s.channels;   // (with 16-byte pieces: where the first does)
        span = (long long)(kGroups * N) * csize * times;
        t0 = (long long)((int)rank * times + time) * (kGroups * N);
        off = lane / 8 * N;
        rounds = (int)((s.steps + span - 1) / span);
    }
};

// The resets of a warp's tile, a step or two a lane: requested a tile ahead, used as bits of a lane's own steps.
struct Resets {
    unsigned lo, hi;
};

template <int N>
__device__ __forceinline__ Resets request_resets(const ScanArgs &s, long long b, long long t0)
{
    Resets r{0, 0};
    if (!s.resets) return r;
    const int lane = threadIdx.x & 31;
    const uint8_t *p = s.resets + b * s.sr[0] + (t0 + lane) * s.sr[1];
    if (t0 + lane < s.steps) r.lo = *p;
    if (kGroups * N > 32 && t0 + 32 + lane < s.steps) r.hi = p[32 * s.sr[1]];
    return r;
}

template <int N>
__device__ __forceinline__ unsigned reset_bits(Resets r)
{
    const unsigned a = __ballot_sync(kFull, r.lo != 0);
    const int first = (threadIdx.x & 31) / 8 * N;   // of the tile's steps
    if constexpr (kGroups * N > 32) {
        const unsigned c = __ballot_sync(kFull, r.hi != 0);
        return (first < 32 ? a : c) >> (first & 31) & ((1u << N) - 1u);
    }
    return a >> first & ((1u << N) - 1u);
}

template <int N>
__device__ __forceinline__ F2 first_state(const float *p, const ScanArgs &s, const Place<N> &me)
{
    const long long i = me.b * s.channels + me.ch;
    return {p && me.live ? p[i] : 0.0f, p && me.second ? p[i + 1] : 0.0f};
}

template <int N>
__device__ __forceinline__ void last_state(float *p, F2 v, const ScanArgs &s, const Place<N> &me)
{
    if (!p || me.rank != 0 || (threadIdx.x & 31) >= 8) return;
    const long long i = me.b * s.channels + me.ch;
    if (me.live) p[i] = v.x;
    if (me.second) p[i + 1] = v.y;
}

// A tile between its two sweeps.
template <int N, int NV>
struct Held {
    F2 w[N], v[NV];
    Stretch before[2], all[2];
    unsigned resets;
    bool plain, any;   // any: a lane of the warp has resets
};

// Whether a lane's products and sums can be taken as they are: check is 0 then, A is neither 0 nor NaN, and H is
// finite.  A channel that does not exist passes its state on.
template <int N>
__device__ __forceinline__ bool settle(F2 &A, F2 &H, F2 check, const Place<N> &me, bool whole)
{
    if (!me.second) {
        A.y = 1.0f;
        H.y = check.y = 0.0f;
        if (!me.live) {
            A.x = 1.0f;
            H.x = 0.0f;
            return true;
        }
    }
    return whole && fabsf(A.x) > 0.0f && fabsf(A.y) > 0.0f && fabsf(H.x) < kInf && fabsf(H.y) < kInf && check.x == 0.0f &&
           check.y == 0.0f;
}

// (Neither kernel lets the next one begin before it ends: the next one's CTAs would take the few places that are free
// meanwhile and lie unevenly on the SMs.  Both passes of 8 x 16384 x 1024 f32 take 742 us; with the release at the
// kernels' end 786, at their start 881.)
//
// Each sweep is first written with products and sums alone: w h + v, and a reset's state of 0 by a select
// where a warp has any.  That is right unless a weight is 0 (then the product A is, or may be) or a dropped
// input is not finite (then H is not), or not every step exists; those lanes go the careful way.
template <typename T, int N, bool SIG, bool WIDE, bool CLUSTER, int ST>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) k_scan_fwd(ScanArgs s, unsigned ctiles, unsigned csize, int times)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    // Alone, a warp keeps a tile's weights and inputs in registers from one sweep to the next, and the tile's place
    // is free after the first.  With a cluster two tiles are under way, which would take too many: the second
    // sweep works them out again.
    constexpr bool HOLD = !CLUSTER;
    constexpr int AHEAD = CLUSTER ? ST - 2 : ST - 1;
    typedef Ring<T, N, 2, ST, WIDE> R;
    const Place<N> me(s, ctiles, csize, times);
    const R ring{dyn + (threadIdx.x >> 5) * R::BYTES};
    Joints<CLUSTER> joints;
    pdl_wait();
    const T *a = static_cast<const T *>(s.a) + me.b * s.sa[0] + me.c0;
    const T *x = static_cast<const T *>(s.x) + me.b * s.sx[0] + me.c0;
    T *out = static_cast<T *>(s.out_h) + me.b * s.sh[0] + me.ch;
    auto request = [&](int k) {
        ring.request(k, 0, a, s.sa[1], me.t0 + k * me.span, s.steps, me.channels);
        ring.request(k, 1, x, s.sx[1], me.t0 + k * me.span, s.steps, me.channels);
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < (CLUSTER ? AHEAD : ST); ++k) request(k);
    Resets ahead = request_resets<N>(s, me.b, me.t0);
    joints.state = first_state(s.h0, s, me);
    joints.begin(s, dyn + (blockDim.x >> 5) * R::BYTES, me.strip, times, me.time, csize, me.rank);

    typedef Held<HOLD ? N : 1, HOLD ? N : 1> Tile;
    auto weights = [&](int k, int i, F2 &w, F2 &v) {
        w = ring.read(k, 0, i);
        v = ring.read(k, 1, i);
        if constexpr (SIG) {
            F2 c;
            gates<T>(w, w, c);
            v = v * c;
        }
    };
    // the same with care; past the end the state stays
    auto weights_of = [&](int k, int i, int c, bool valid, bool reset, float &w, float &v) {
        w = 1.0f;
        v = 0.0f;
        if (!valid) return;
        const Gate g = gate<T, SIG>(at(ring.read(k, 0, i), c));
        v = at(ring.read(k, 1, i), c);
        v = SIG ? weigh(g.v, v, 0.0f) : v;
        w = reset ? 0.0f : g.w;
    };
    auto first = [&](int k, Tile &h) {
        const long long t = me.t0 + k * me.span + me.off;
        copies_wait<CLUSTER ? AHEAD - 1 : AHEAD>();
        __syncwarp();
        if (CLUSTER) request(k + AHEAD);   // (the place was last read before this warp's last shuffles)
        const unsigned resets = reset_bits<N>(ahead);
        ahead = request_resets<N>(s, me.b, t - me.off + me.span);
        h.resets = resets;
        F2 A{1.0f, 1.0f}, H{0.0f, 0.0f};
        F2 check{0.0f, 0.0f};   // NaN once an input is not finite: its weight of 0 may have to drop it, and a reset hides it
        auto run = [&](auto any) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                F2 w, v;
                weights(k, i, w, v);
                if constexpr (SIG && any.value) check = fma2(v, F2{0.0f, 0.0f}, check);
                if constexpr (HOLD) {
                    h.w[i] = w;
                    h.v[i] = v;
                }
                if (any.value && resets >> i & 1u) H = {0.0f, 0.0f};
                H = fma2(w, H, v);
                A = A * w;
            }
        };
        h.any = __any_sync(kFull, resets != 0);
        if (h.any) run(std::true_type());
        else run(std::false_type());
        Stretch own[2];
        h.plain = settle(A, H, check, me, t + N <= s.steps);
        if (!h.plain) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                own[c] = {1.0f, 0.0f};
                bool drop = false;
#pragma unroll HOLD ? N : 1
                for (int i = 0; i < N; ++i) {
                    float w, v;
                    weights_of(k, i, c, (c ? me.second : me.live) && t + i < s.steps, resets >> i & 1u, w, v);
                    if constexpr (HOLD) {
                        at(h.w[i], c) = w;
                        at(h.v[i], c) = v;
                    }
                    drop = drop || w == 0.0f;
                    own[c].H = weigh(w, own[c].H, v);
                    own[c].A *= w;
                }
                own[c].A = drop ? __int_as_float(0x7fffffff) : nonzero(own[c].A);
            }
        } else {
            const float nan = __int_as_float(0x7fffffff);
            own[0] = {resets && me.live ? nan : A.x, H.x};
            own[1] = {resets && me.second ? nan : A.y, H.y};
        }
        joints.first(k, h.plain, A, H, resets != 0, own, h.before, h.all);
        if (!CLUSTER) {
            __syncwarp();   // every lane has read the tile
            request(k + ST);
        }
    };
    auto second = [&](int k, const Tile &h) {
        const long long t = me.t0 + k * me.span + me.off;
        F2 st = joints.second(s, k, h.before, h.all);
        const long long stride = s.sh[1];
        T *o = out + t * stride;
        if (!me.live) {
            // nothing to store
        } else if (h.plain) {
            auto run = [&](auto any) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    F2 w, v;
                    if constexpr (HOLD) {
                        w = h.w[i];
                        v = h.v[i];
                    } else {
                        weights(k, i, w, v);
                    }
                    if (any.value && h.resets >> i & 1u) st = {0.0f, 0.0f};
                    st = fma2(w, st, v);
                    store2<T, WIDE>(o + i * stride, st, me.second);
                }
            };
            if (h.any) run(std::true_type());
            else run(std::false_type());
        } else {
#pragma unroll HOLD ? N : 1
            for (int i = 0; i < N; ++i) {
                if (t + i >= s.steps) break;
                F2 w, v;
                if constexpr (HOLD) {
                    w = h.w[i];
                    v = h.v[i];
                } else {
                    weights_of(k, i, 0, true, h.resets >> i & 1u, w.x, v.x);
                    weights_of(k, i, 1, me.second, h.resets >> i & 1u, w.y, v.y);
                }
                st = {weigh(w.x, st.x, v.x), weigh(w.y, st.y, v.y)};
                store2<T, WIDE>(o + i * stride, st, me.second);
            }
        }
    };
    if constexpr (CLUSTER) {
        // (one copy of each sweep: the code has to stay in the caches)
        Tile now{}, before{};
        for (int k = 0; k <= me.rounds; ++k) {
            if (k < me.rounds) first(k, now);
            if (k > 0) second(k - 1, before);
            before = now;
        }
    } else {
        Tile h;
        for (int k = 0; k < me.rounds; ++k) {
            first(k, h);
            second(k, h);
        }
    }
    joints.end(s);
    if (me.time == 0) last_state(s.last, joints.state, s, me);
}

// The gradient, on arrays turned so that step 0 is the last one forward; s.h is shifted by one step, so
// that row t holds the state before that step (row steps - 1 is h0).
template <typename T, int N, bool SIG, bool WIDE, bool CLUSTER, int ST>
__global__ void __launch_bounds__(kWarps * 32, CLUSTER ? kCtasPerSmBack : kCtasPerSm) k_scan_bwd(ScanArgs s, unsigned ctiles, unsigned csize, int times)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int NA = SIG ? 4 : 3;
    constexpr bool HOLD = !CLUSTER;
    constexpr int AHEAD = CLUSTER ? ST - 2 : ST - 1;   // with a cluster the tile before is still read
    typedef Ring<T, N, NA, ST, WIDE> R;
    const Place<N> me(s, ctiles, csize, times);
    const R ring{dyn + (threadIdx.x >> 5) * R::BYTES};
    Joints<CLUSTER> joints;
    pdl_wait();
    const T *a = static_cast<const T *>(s.a) + me.b * s.sa[0] + me.c0;
    const T *gh = static_cast<const T *>(s.gh) + me.b * s.sgh[0] + me.c0;
    const T *h = static_cast<const T *>(s.h) + me.b * s.sh[0] + me.c0;
    const T *x = SIG ? static_cast<const T *>(s.x) + me.b * s.sx[0] + me.c0 : nullptr;
    T *ga = s.ga ? static_cast<T *>(s.ga) + me.b * s.sga[0] + me.ch : nullptr;
    T *gx = s.gx ? static_cast<T *>(s.gx) + me.b * s.sgx[0] + me.ch : nullptr;
    auto request = [&](int k) {
        const long long t = me.t0 + k * me.span;
        ring.request(k, 0, a, s.sa[1], t, s.steps, me.channels);
        ring.request(k, 1, gh, s.sgh[1], t, s.steps, me.channels);
        ring.request(k, 2, h, s.sh[1], t, s.steps - 1, me.channels);
        if (SIG) ring.request(k, 3, x, s.sx[1], t, s.steps, me.channels);
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) request(k);
    Resets ahead = request_resets<N>(s, me.b, me.t0);
    joints.state = first_state(s.glast, s, me);
    joints.begin(s, dyn + (blockDim.x >> 5) * R::BYTES, me.strip, times, me.time, csize, me.rank);

    typedef Held<HOLD ? N : 1, HOLD && SIG ? N : 1> Tile;
    auto first = [&](int k, Tile &d) {
        const long long t = me.t0 + k * me.span + me.off;
        copies_wait<CLUSTER ? AHEAD - 1 : AHEAD>();
        __syncwarp();
        if (CLUSTER) request(k + AHEAD);   // (the place was last read before this warp's last shuffles)
        const unsigned resets = reset_bits<N>(ahead);
        ahead = request_resets<N>(s, me.b, t - me.off + me.span);
        d.resets = resets;
        F2 A{1.0f, 1.0f}, H{0.0f, 0.0f};
        auto run = [&](auto any) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                F2 w = ring.read(k, 0, i), v;
                if constexpr (SIG) gates<T>(w, w, v);
                if constexpr (HOLD) d.w[i] = w;
                if constexpr (HOLD && SIG) d.v[i] = v;
                H = w * (H + ring.read(k, 1, i));
                if (any.value && resets >> i & 1u) H = {0.0f, 0.0f};
                A = A * w;
            }
        };
        d.any = __any_sync(kFull, resets != 0);
        if (d.any) run(std::true_type());
        else run(std::false_type());
        Stretch own[2];
        d.plain = settle(A, H, F2{0.0f, 0.0f}, me, t + N < s.steps);   // (row steps - 1 reads h0)
        if (d.plain) {
            const float nan = __int_as_float(0x7fffffff);
            own[0] = {resets && me.live ? nan : A.x, H.x};
            own[1] = {resets && me.second ? nan : A.y, H.y};
        }
        if (!d.plain) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                own[c] = {1.0f, 0.0f};
                bool drop = false;
#pragma unroll 1
                for (int i = 0; i < N; ++i) {
                    if (!((c ? me.second : me.live) && t + i < s.steps)) break;
                    const float w = resets >> i & 1u ? 0.0f : gate<T, SIG>(at(ring.read(k, 0, i), c)).w;
                    drop = drop || w == 0.0f;
                    own[c].H = weigh(w, own[c].H + at(ring.read(k, 1, i), c), 0.0f);
                    own[c].A *= w;
                }
                own[c].A = drop ? __int_as_float(0x7fffffff) : nonzero(own[c].A);
            }
        }
        joints.first(k, d.plain, A, H, resets != 0, own, d.before, d.all);
    };
    auto second = [&](int k, const Tile &d) {
        const long long t = me.t0 + k * me.span + me.off;
        F2 c = joints.second(s, k, d.before, d.all);
        const F2 start = c;
        const long long stride_a = s.sga[1], stride_x = s.sgx[1];
        T *oa = ga + t * stride_a, *ox = gx + t * stride_x;
        bool plain = d.plain || !me.live;
        if (plain && me.live) {
            F2 check{0.0f, 0.0f};   // NaN once a gradient is not finite: a slope of 0 may have to drop it
            auto run = [&](auto any) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const bool reset = any.value && (d.resets >> i & 1u);
                    const F2 g = ring.read(k, 1, i) + c;
                    F2 before = ring.read(k, 2, i), da, dx, w, v;
                    if constexpr (HOLD) {
                        w = d.w[i];
                        if constexpr (SIG) v = d.v[i];
                    } else {
                        w = ring.read(k, 0, i);
                        if constexpr (SIG) gates<T>(w, w, v);
                    }
                    if (reset) before = {0.0f, 0.0f};
                    if constexpr (SIG) {
                        da = g * fma2(ring.read(k, 3, i), F2{-1.0f, -1.0f}, before) * (w * v);
                        dx = g * v;
                        check = fma2(da, F2{0.0f, 0.0f}, check);
                    } else {
                        da = g * before;
                        dx = g;
                        if (reset) da = {0.0f, 0.0f};
                    }
                    c = w * g;
                    if (reset) c = {0.0f, 0.0f};
                    if (ga) store2<T, WIDE>(oa + i * stride_a, da, me.second);
                    if (gx) store2<T, WIDE>(ox + i * stride_x, dx, me.second);
                }
            };
            if (d.any) run(std::true_type());
            else run(std::false_type());
            plain = !SIG || (check.x == 0.0f && (check.y == 0.0f || !me.second));
        }
        if (!plain) {
            const F2 h0 = first_state(s.h0, s, me);
            c = start;
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                if (!(me.live && t + i < s.steps)) break;
                const bool reset = d.resets >> i & 1u;
                const F2 rw = ring.read(k, 0, i), rg = ring.read(k, 1, i);
                const F2 rb = t + i == s.steps - 1 ? h0 : ring.read(k, 2, i);
                const F2 rx = SIG ? ring.read(k, 3, i) : F2{0.0f, 0.0f};
                F2 da, dx;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Gate f = gate<T, SIG>(at(rw, e));
                    const float g = at(rg, e) + at(c, e), before = reset ? 0.0f : at(rb, e);
                    if (SIG) {
                        const float slope = f.w * f.v;
                        at(da, e) = slope == 0.0f ? 0.0f : g * (before - at(rx, e)) * slope;
                        at(dx, e) = weigh(f.v, g, 0.0f);
                    } else {
                        at(da, e) = reset ? 0.0f : g * before;
                        at(dx, e) = g;
                    }
                    at(c, e) = weigh(reset ? 0.0f : f.w, g, 0.0f);
                }
                if (ga) store2<T, WIDE>(oa, da, me.second);
                if (gx) store2<T, WIDE>(ox, dx, me.second);
                oa += s.sga[1];
                ox += s.sgx[1];
            }
        }
        if (!CLUSTER) {
            __syncwarp();   // every lane has read the tile
            request(k + ST);
        }
    };
    if constexpr (CLUSTER) {
        Tile now{}, before{};
        for (int k = 0; k <= me.rounds; ++k) {
            if (k < me.rounds) first(k, now);
            if (k > 0) second(k - 1, before);
            before = now;
        }
    } else {
        Tile d;
        request(ST - 1);
        for (int k = 0; k < me.rounds; ++k) {
            first(k, d);
            second(k, d);
        }
    }
    joints.end(s);
    if (me.time == 0) last_state(s.gh0, joints.state, s, me);
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

// Many channels or few steps: one thread takes VEC channels through all steps, some rows requested ahead.  The
// least instructions, and HBM's rate where the channels alone keep enough bytes in flight (512 x 64 x 4096
// bf16 sigmoid: forward 94% of the copy rate).
constexpr int kFewAhead = 8, kFewAheadBack = 4;

template <typename T, bool SIG, int VEC>
__global__ void __launch_bounds__(128) k_scan_few(ScanArgs s)
{
    typedef Cell<T, VEC> C;
    typedef typename C::Raw Raw;
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
    const uint8_t *resets = s.resets ? s.resets + b * s.sr[0] : nullptr;
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = s.h0 ? s.h0[b * s.channels + ch + e] : 0.0f;
    for (long long t = 0; t < s.steps; t += kFewAhead) {
        Raw ra[kFewAhead], rx[kFewAhead];
        bool reset[kFewAhead];
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) {
            if (t + i >= s.steps) continue;
            ra[i] = *reinterpret_cast<const Raw *>(a + (t + i) * s.sa[1]);
            rx[i] = *reinterpret_cast<const Raw *>(x + (t + i) * s.sx[1]);
            reset[i] = resets && resets[(t + i) * s.sr[1]];
        }
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) {
            if (t + i >= s.steps) continue;
            float w[VEC], v[VEC];
            C::unpack(ra[i], w);
            C::unpack(rx[i], v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const Gate g = gate<T, SIG>(w[e]);
                h[e] = weigh(reset[i] ? 0.0f : g.w, h[e], SIG ? weigh(g.v, v[e], 0.0f) : v[e]);
            }
            C::store(out + (t + i) * s.sh[1], h);
        }
    }
    if (s.last) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) s.last[b * s.channels + ch + e] = h[e];
    }
}

// The gradient of the same, on the turned arrays (as k_scan_bwd).
template <typename T, bool SIG, int VEC>
__global__ void __launch_bounds__(128) k_scan_few_bwd(ScanArgs s)
{
    typedef Cell<T, VEC> C;
    typedef typename C::Raw Raw;
    const unsigned per = s.channels / VEC;
    const unsigned id = blockIdx.x * 128 + threadIdx.x;
    pdl_wait();
    pdl_release();
    if (id >= per * s.batch) return;
    const long long b = id / per;
    const unsigned ch = id % per * VEC;
    const T *a = static_cast<const T *>(s.a) + b * s.sa[0] + ch;
    const T *gh = static_cast<const T *>(s.gh) + b * s.sgh[0] + ch;
    const T *h = static_cast<const T *>(s.h) + b * s.sh[0] + ch;
    const T *x = SIG ? static_cast<const T *>(s.x) + b * s.sx[0] + ch : nullptr;
    T *ga = s.ga ? static_cast<T *>(s.ga) + b * s.sga[0] + ch : nullptr;
    T *gx = s.gx ? static_cast<T *>(s.gx) + b * s.sgx[0] + ch : nullptr;
    const uint8_t *resets = s.resets ? s.resets + b * s.sr[0] : nullptr;
    float c[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) c[e] = s.glast ? s.glast[b * s.channels + ch + e] : 0.0f;
    for (long long t = 0; t < s.steps; t += kFewAheadBack) {
        Raw ra[kFewAheadBack], rg[kFewAheadBack], rh[kFewAheadBack], rx[SIG ? kFewAheadBack : 1];
        bool reset[kFewAheadBack];
#pragma unroll
        for (int i = 0; i < kFewAheadBack; ++i) {
            if (t + i >= s.steps) continue;
            ra[i] = *reinterpret_cast<const Raw *>(a + (t + i) * s.sa[1]);
            rg[i] = *reinterpret_cast<const Raw *>(gh + (t + i) * s.sgh[1]);
            if (t + i < s.steps - 1) rh[i] = *reinterpret_cast<const Raw *>(h + (t + i) * s.sh[1]);
            if constexpr (SIG) rx[i] = *reinterpret_cast<const Raw *>(x + (t + i) * s.sx[1]);
            reset[i] = resets && resets[(t + i) * s.sr[1]];
        }
#pragma unroll
        for (int i = 0; i < kFewAheadBack; ++i) {
            if (t + i >= s.steps) continue;
            float w[VEC], g[VEC], before[VEC], da[VEC], dx[VEC];
            C::unpack(ra[i], w);
            C::unpack(rg[i], g);
            if constexpr (SIG) C::unpack(rx[i], dx);
            if (t + i < s.steps - 1) {
                C::unpack(rh[i], before);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) before[e] = s.h0 ? s.h0[b * s.channels + ch + e] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const Gate f = gate<T, SIG>(w[e]);
                const float gt = g[e] + c[e], bt = reset[i] ? 0.0f : before[e];
                if (SIG) {
                    const float slope = f.w * f.v;
                    da[e] = slope == 0.0f ? 0.0f : gt * (bt - dx[e]) * slope;
                    dx[e] = weigh(f.v, gt, 0.0f);
                } else {
                    da[e] = reset[i] ? 0.0f : gt * bt;
                    dx[e] = gt;
                }
                c[e] = weigh(reset[i] ? 0.0f : f.w, gt, 0.0f);
            }
            if (ga) C::store(ga + (t + i) * s.sga[1], da);
            if (gx) C::store(gx + (t + i) * s.sgx[1], dx);
        }
    }
    if (s.gh0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) s.gh0[b * s.channels + ch + e] = c[e];
    }
}

// ---- launches --------------------------------------------------------------------------------

// How a pass is laid out: a CTA of `strips` x `times` warps, clusters of csize CTAs.
struct Layout {
    int strips, times;
    unsigned csize;
    unsigned warps() const { return (unsigned)(strips * times); }
};

template <typename T, bool SIG, bool WIDE, bool BACK, bool CLUSTER>
struct Launch {
    static constexpr int NA = BACK ? (SIG ? 4 : 3) : 2, ST = CLUSTER ? kRingCluster : kRing;
    static constexpr int N = CLUSTER && sizeof(T) == 2 ? kLaneStepsCluster16 : kLaneSteps, TILE = kGroups * N;
    static auto kernel()
    {
        if constexpr (BACK) return k_scan_bwd<T, N, SIG, WIDE, CLUSTER, ST>;
        else return k_scan_fwd<T, N, SIG, WIDE, CLUSTER, ST>;
    }
    static size_t smem(const Layout &l)
    {
        return l.strips * (l.times * (size_t)Ring<T, N, NA, ST, WIDE>::BYTES + Joints<CLUSTER>::bytes(l.times, l.csize));
    }
    // CTAs that run at once: asked once for each layout and device (0: not asked yet)
    static cudaError_t capacity(const Layout &l, const DeviceInfo &dev, int *ctas)
    {
        static std::atomic<int> known[64][3][3][5];
        auto log2of = [](unsigned v) { return v >= 16 ? 4 : v >= 8 ? 3 : v >= 4 ? 2 : v >= 2 ? 1 : 0; };
        std::atomic<int> &k = known[dev.device][log2of(l.strips)][log2of(l.times)][log2of(l.csize)];
        *ctas = k.load(std::memory_order_relaxed);
        if (*ctas) return cudaSuccess;
        cudaError_t e = cudaFuncSetAttribute(kernel(), cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel(), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess && l.csize == 1) {
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, kernel(), l.warps() * 32, smem(l));
            *ctas *= dev.sms;
        } else if (e == cudaSuccess) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(l.csize);
            cfg.blockDim = dim3(l.warps() * 32);
            cfg.dynamicSmemBytes = smem(l);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = l.csize;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(ctas, kernel(), &cfg);
            *ctas *= (int)l.csize;
        }
        if (e == cudaSuccess && *ctas <= 0) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess) k.store(*ctas, std::memory_order_relaxed);
        return e;
    }
    static cudaError_t run(const ScanArgs &a, const Layout &l, cudaStream_t st)
    {
        const unsigned ctiles = (a.channels + kStrip * l.strips - 1) / (kStrip * l.strips);
        const unsigned long long grid = (unsigned long long)ctiles * a.batch * l.csize;
        if (grid > 0x7fffffffull) return cudaErrorInvalidConfiguration;
        return launch_clusters(kernel(), (unsigned)grid, l.warps() * 32, l.csize, smem(l), st, a, ctiles, l.csize, l.times);
    }
};

// What a pass is laid out as: the one that should finish first by a model whose constants are measured.
// Tiles: a round of an SM takes the time of its bytes at HBM's rate (times `tile_cost`: 64 x 1024 x 1024 bf16
// 80 us against 60, binary32 120 against 119, single values 333 against 118), or what one warp's round takes
// by itself, whichever is longer (0.8 us, with a CTA barrier 1.0, with a cluster's exchange 2.5); CTAs beyond
// what fits at once run after the others.  One thread a channel through all steps: `flat` us a step for
// the latency of its rows and their bytes at HBM's rate (1 x 1024 x 256 bf16: 185 us, as tiles 5; 64 x 4 x 4096:
// 3.6 us, as tiles 25).
template <typename T, bool SIG, bool WIDE, bool BACK>
cudaError_t launch_any(const ScanArgs &a, const DeviceInfo &dev, cudaStream_t st)
{
    typedef Launch<T, SIG, WIDE, BACK, false> One;
    typedef Launch<T, SIG, WIDE, BACK, true> Many;
    const unsigned per_row = (a.channels + kStrip - 1) / kStrip;
    constexpr double step_us = kStrip * sizeof(T) * (One::NA + (BACK ? 2 : 1)) / 44500.0;   // of a warp's strip
    Layout best{};
    constexpr int P = WIDE ? 16 / (int)sizeof(T) : 1;
    const double cells = (double)a.channels * a.batch;
    constexpr double flat = WIDE ? (BACK ? 0.25 : 0.13) : (BACK ? 0.4 : 0.27);
    constexpr double tile_cost = !WIDE ? 2.2 : sizeof(T) == 4 ? 1.05 : 1.35;
    const double few = a.steps * (flat + cells * sizeof(T) * (One::NA + (BACK ? 2 : 1)) / 6.4e6);
    double least = 1e30;
    for (int times = 1; times <= 4; times *= 2) {
        for (unsigned csize = 1; csize <= (times == 4 ? (unsigned)kMaxCluster : 1u); csize *= 2) {
            const int tile = csize > 1 ? Many::TILE : One::TILE;
            const long long span = (long long)tile * times * csize;
            if (times * csize > 1 && span / 2 >= a.steps) continue;   // some would have no tile
            Layout l{1, times, csize};
            while (l.strips * 2 * times <= 4 && (unsigned)l.strips < per_row) l.strips *= 2;
            int fit = 0;
            const cudaError_t e = csize > 1 ? Many::capacity(l, dev, &fit) : One::capacity(l, dev, &fit);
            if (e != cudaSuccess) return e;
            const double ctas = (double)((per_row + l.strips - 1) / l.strips) * a.batch * csize;
            const double alone = csize > 1 ? 2.5 : times > 1 ? 1.0 : 0.8;
            const double full = std::floor(ctas / fit), rest = ctas - full * fit;
            auto round = [&](double n) { return std::max(alone, n / dev.sms * l.warps() * tile * step_us); };
            const double us = std::ceil((double)a.steps / span) * (full * round(fit) + (rest > 0 ? round(rest) : 0.0));
            if (us < least) {
                least = us;
                best = l;
            }
        }
    }
    if (few <= least * tile_cost + 3.0) {
        const unsigned grid = (unsigned)((unsigned long long)(a.channels / P) * a.batch + 127) / 128;
        if constexpr (BACK) return launch_clusters(k_scan_few_bwd<T, SIG, P>, grid, 128, 1, 0, st, a);
        else return launch_clusters(k_scan_few<T, SIG, P>, grid, 128, 1, 0, st, a);
    }
    return best.csize > 1 ? Many::run(a, best, st) : One::run(a, best, st);
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
    return wide ? launch_any<T, SIG, true, false>(a, dev, st) : launch_any<T, SIG, false, false>(a, dev, st);
}

template <typename T, bool SIG>
cudaError_t bwd_t(const ScanArgs &a, const DeviceInfo &dev, cudaStream_t st)
{
    constexpr unsigned e = sizeof(T), P = 16 / e;
    const bool wide = a.channels % P == 0 && aligned16(a.a, a.sa, a, e) && aligned16(a.x, a.sx, a, e) &&
                      aligned16(a.h, a.sh, a, e) && aligned16(a.gh, a.sgh, a, e) && aligned16(a.ga, a.sga, a, e) &&
                      aligned16(a.gx, a.sgx, a, e);
    return wide ? launch_any<T, SIG, true, true>(a, dev, st) : launch_any<T, SIG, false, true>(a, dev, st);
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
