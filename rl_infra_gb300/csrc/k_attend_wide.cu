// k_attend_wide.cu -- attention over a paged cache for many rows: the products on the tensor cores' own
// instruction, with scores, p and outputs in tensor memory.
//
// A head of keys with many rows (query heads times nodes) is bound by its products, which the warp-wide
// instruction makes at a quarter of the rate.  Here one thread issues them on tiles of 128 rows by 128 keys;
// another warp asks the copy engine for keys and values (a ring of tiles, keys and values in turn); two groups of
// four warps take the softmax, a thread a row.  Each group has its scores and its output in tensor memory:
//     up to 128 rows:  both groups take the same rows and every other tile of keys, and join at the end;
//     more:            each group takes 128 of up to 256 rows, and both every tile.
// While one group turns scores into p (written over them, rounded to the type), the other's products run.
//
// The maximum that p refers to is raised only where a row's rises by more than 2^8 (float16: 2^4; exact all the same: p and
// its sums keep their relative precision, and stay below 2^16 x 2^31): outputs in tensor memory are then
// scaled, which is rare.  So p is worked out in one pass over the scores, which also finds their maximum; where that
// has risen, the pass is made again.
//
// Measured (GB300): 32 trees of 64 nodes, 64 query heads on 8, up to 6000 tokens, bf16 288 us, 920 TFLOP/s (a chain of
// the softmax, 1250 cycles a tile of 128 x 128, and two products of 512 each, while the other group does the same; the
// tensor cores are busy half of the time); 16 trees of 24 nodes, 96 rows a head of 64 entries, up to 8000 tokens, f16 57 us,
// 3.36 TB/s.  With the warp-wide instruction 1611 and 236 us.
//
// What was tried and not kept: registers dealt anew between the warps (setmaxnreg; the compiler then spilled 2.4 KB a
// thread: 2309 us); outputs by way of shared memory, mask bytes asked for without branches, a warp without rows that skips
// its softmax (297 to 312 us of GPU time, at 286 without each: the loop's registers are full, and it spills); a second way
// through the loop for scores past kFar, as a call or in place (304 and 317 us, at 284 without).
#include "attend_mma.cuh"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace gbper {
namespace attend {
namespace {

constexpr int kGroups = 2, kThreads = kGroups * 128 + 96;   // and two warps for the copies, one for the products
constexpr unsigned kBegin = 6;                               // tiles that a sequence's begin and end are worth
constexpr int KT = 128;                                      // keys of a tile, and rows of a group
// What a row's maximum may rise above the one that p refers to, in log2, and what p = 2^(s - top + kUp) has there: a float16
// uses its upper end too (p up to 2^15.5), for what `below` in attend_mma.cuh says: 11 bits down
// to 2^-25.5 of the maximum, off by at most 2^-36.5 of it below.  Each rise costs a second pass over a tile's scores: with 2
// and 13 there were so many that 32 trees of 64 nodes took 371 us, with 4 284 us, as with 8.
template <typename T> constexpr float kRise = std::is_same<T, __half>::value ? 4.0f : 8.0f;
template <typename T> constexpr float kUp = std::is_same<T, __half>::value ? 11.5f : 0.0f;
constexpr int kColumns = 512;                                // of tensor memory: two of scores, two of outputs, 128 each

template <bool PAIR>
struct Tail {
    u64 full[10], empty[10], q_ready, s_full[2], p_ready[2], o_full[2], meet, last;
    u64 scan[kThreads / 32];
    unsigned bad[10][4];
    alignas(16) int boxes[2][KT];
    float ml[PAIR ? 1 : 256][2];   // maxima and sums, where both groups have the same rows
    unsigned asked[2];             // the numbers of the next tiles that the warps would have asked for
    unsigned dead[2], odd, tmem;   // whether a wait gave up, and their limit
};

template <int DP, bool PAIR>
struct Cfg {
    static constexpr int TILE = KT * DP * 2;                 // bytes of a tile of keys or of values
    static constexpr int QB = (PAIR ? 2 : 1) * TILE;
    static constexpr int TAIL = ((int)sizeof(Tail<PAIR>) + 63) / 64 * 64;
    static constexpr int FIT = (227 * 1024 - QB - TAIL) / TILE;
    static constexpr int ST = FIT > 10 ? 10 : FIT;
    static constexpr int SMEM = ST * TILE + QB + TAIL;
    static constexpr int M = PAIR ? 256 : 128;
    static_assert(ST >= 5, "the keys of the next tile come before this one's values are free");
};

// ---- the tensor cores' instructions ---------------------------------------------------------------
// Operands of 128-byte rows, 16-byte pieces turned modulo 8; groups of 8 rows 1024 bytes apart.  `lead`: bytes
// between blocks of 64 entries where those run across the product's columns (values).
__device__ __forceinline__ u64 operand(unsigned at, unsigned lead)
{
    return (u64)((at & 0x3ffffu) >> 4) | (u64)(lead >> 4) << 16 | (u64)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// 128 rows by n columns, binary32 sums; b_wide: the second operand's entries run along its columns
template <typename T>
__host__ __device__ constexpr unsigned product(unsigned n, bool b_wide)
{
    return 1u << 4 | (std::is_same<T, __nv_bfloat16>::value ? 1u << 7 | 1u << 10 : 0u) | (b_wide ? 1u << 16 : 0u) | (n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void multiply(unsigned d, u64 a, u64 b, unsigned how, unsigned add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(how), "r"(add) : "memory");
}
__device__ __forceinline__ void multiply_t(unsigned d, unsigned a, u64 b, unsigned how, unsigned add)   // a in tensor memory
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(how), "r"(add) : "memory");
}
// arrives when all products issued before are done
__device__ __forceinline__ void commit(unsigned bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// (names what was loaded, so that nothing that reads it is moved before the wait)
#define KEEP32(v) "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), \
    "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), \
    "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), \
    "+f"(v[30]), "+f"(v[31])
__device__ __forceinline__ void loaded32(float *v) { asm volatile("" : KEEP32(v)::"memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define REGS32(v) "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), \
    "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), \
    "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), \
    "=f"(v[30]), "=f"(v[31])
// 32 columns of a warp's 32 lanes, a thread a lane
__device__ __forceinline__ void get32(float *v, unsigned at)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
                 "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];" : REGS32(v) : "r"(at) : "memory");
}
#define ARGS32(v) "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), \
    "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), \
    "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
__device__ __forceinline__ void put32(unsigned at, const float *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::ARGS32(v), "r"(at) : "memory");
}
#define WORDS32(v) "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), \
    "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), \
    "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
__device__ __forceinline__ void put32(unsigned at, const unsigned *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::WORDS32(v), "r"(at) : "memory");
}

// A reference past kFar in log2 cannot stay one: p = 2^(s c2 - top) carries its rounding, up to a quarter there (what float16's
// range has room for) and 128 at 2^31, as much as binary32 holds.  What such a row refers to is taken off its scores
// themselves, in tensor memory.
constexpr float kFar = 4194304.0f;
__device__ __forceinline__ void take_off(unsigned my_s, float shift)
{
#pragma unroll 1
    for (unsigned i = 0; i < KT / 32; ++i) {
        float sc[32];
        get32(sc, my_s + 32 * i);
        wait_ld();
        loaded32(sc);
#pragma unroll
        for (int k = 0; k < 32; ++k) sc[k] -= shift;
        put32(my_s + 32 * i, sc);
    }
    wait_st();
}

// the scores of 32 keys that are not seen
__device__ __forceinline__ void hide(float *sc, unsigned word)
{
#pragma unroll
    for (int k = 0; k < 32; ++k)
        if (!(word >> k & 1u)) sc[k] = -INFINITY;
}

// bit k of word[k / 32]: the row of node n sees key first + k
__device__ __forceinline__ void seen(const AttendArgs &a, unsigned b, const Span &s, int n, unsigned first, const unsigned *bad,
                                     bool wrong, unsigned shift, unsigned *word)
{
    const int there = s.total - s.len;                                 // nodes that the table has a place for
    const int end = a.mask || n < 0 ? there : min(there, n + 1);       // those that may be seen: from 0 to here
    const uint8_t *mask = a.mask ? a.mask + b * a.sm[0] + (long long)max(n, 0) * a.sm[1] : nullptr;
#pragma unroll
    for (int w = 0; w < KT / 32; ++w) {
        const int j0 = (int)(first + 32 * w) - s.len;                  // the node at the word's first bit; < 0: context
        const int below = min(max(-j0, 0), 32), upto = min(max(end - j0, 0), 32);
        unsigned bits = upto == 32 ? ~0u : (1u << upto) - 1;           // context and nodes up to `end`
        const unsigned context = below == 32 ? ~0u : (1u << below) - 1;
        if (mask && (bits & ~context)) {
            unsigned see = 0;
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if ((bits & ~context) >> k & 1u) see |= mask[j0 + k] != 0 ? 1u << k : 0u;
            bits &= context | see;
        }
        if (wrong)
            for (int k = 0; k < 32; ++k) {
                const unsigned box = (w * 32 + k) >> shift;
                if ((bad[box >> 5] >> (box & 31u)) & 1u) bits &= ~(1u << k);
            }
        word[w] = n < 0 ? 0 : bits;
    }
}

template <typename T, int DP, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
k_attend_wide(const __grid_constant__ CacheMaps maps, AttendArgs a, unsigned row_tiles, unsigned max_teams, FastDiv by_group, unsigned shift)
{
    using C = Cfg<DP, PAIR>;
    constexpr int ST = C::ST, M = C::M, TILE = C::TILE;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *qs = smem + ST * TILE;
    Tail<PAIR> &tail = *reinterpret_cast<Tail<PAIR> *>(qs + C::QB);
    volatile unsigned *dead = tail.dead;
    const unsigned t = threadIdx.x, lane = t & 31u, warp = t >> 5;
    const unsigned cta = blockIdx.x, team = cta / row_tiles, rt = cta - team * row_tiles;
    const unsigned group = by_group.d, row0 = rt * M, dim = a.c.dim, halves = (dim + 63) / 64;
    const unsigned full = smem_u32(tail.full), empty = smem_u32(tail.empty), q_ready = smem_u32(&tail.q_ready);
    const unsigned s_full = smem_u32(tail.s_full), p_ready = smem_u32(tail.p_ready), o_full = smem_u32(tail.o_full);

    if (t == 0) {
        for (int i = 0; i < ST; ++i) {
            bar_init(full + 8 * i, 1 + (a.withhold == (i % 2 ? kValues : kKeys)));   // (of its first turn; ST may be odd)
            bar_init(empty + 8 * i, 1 + (a.withhold == kRelease));
        }
        bar_init(q_ready, kGroups * 4 + (a.withhold == kQueries));
        for (int i = 0; i < 2; ++i) {
            bar_init(s_full + 8 * i, 1 + (a.withhold == kScores));
            bar_init(p_ready + 8 * i, 4 + (a.withhold == kP));
            bar_init(o_full + 8 * i, 1 + (a.withhold == kOutputs));
        }
        bar_init(smem_u32(&tail.meet), kGroups * 4 + (a.withhold == kMeet));
        bar_init(smem_u32(&tail.last), 1);
        tail.dead[0] = 0;
        tail.dead[1] = a.wait_ms;
        tail.odd = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pdl_wait();
    pdl_release();
    int *record = reinterpret_cast<int *>(a.work) + (size_t)cta * kRecord;
    if (a.work && t == 0) record[3] = 0;
    Walk<KT, kBegin> w;
    if (!w.template begin<kThreads>(a, team, max_teams, tail.scan)) return;
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tail.tmem)), "r"(kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const unsigned tmem = tail.tmem;
    // scores of group g at column 128 g (p over them), outputs at 256 + 128 g
    unsigned base = 0;         // tiles asked for before this stretch: keys and values in turn
    unsigned stretch = 0;      // stretches before this one

    if (warp == 8 || warp == 10) {   // the warps that ask for tiles, one of keys, one of values
        const unsigned val = warp == 10;
        const CUtensorMap *map = val ? &maps.v : &maps.k;
        const unsigned char *axes = val ? maps.v_at : maps.k_at;
        Loader<KT> load;
        load.shift = shift;
        load.boxes = tail.boxes[val];
        unsigned asked = val;      // the next tile's number: keys even, values odd
        bool ok = true;
        const bool one = chosen();
        while (ok && w.next(a)) {
            if (row0 >= (unsigned)w.s.count * group) continue;
            load.look_up(a, w.b, w.s, w.tile0);
            for (unsigned tile = w.tile0; tile < w.tile1; ++tile) {
                const unsigned slot = asked % ST;
                if (asked >= (unsigned)ST) ok = __all_sync(0xffffffffu, bar_wait(empty + 8 * slot, (asked / ST - 1) & 1, dead));
                if (!ok) break;
                // (bits of what has no page lie with the values, which are given up after the scores have been read)
                load.hand(a, w.s, tile, val ? tail.bad[slot] : nullptr, rt == 0 && w.h == 0);
                if (one) load.template request<DP / 64>(a, map, axes, tile, w.h, smem_u32(smem + slot * TILE), halves, 64, full + 8 * slot);
                asked += 2;
                if (tile + 1 < w.tile1) load.look_up(a, w.b, w.s, tile + 1);
            }
        }
        if (lane == 0) tail.asked[val] = asked;
    } else if (warp == 9) {    // the thread that issues the products
        if (chosen()) {
            const unsigned ksteps = (dim + 15) / 16, q_at = smem_u32(qs);
            unsigned ready[2] = {0, 0};   // phases of p_ready
            bool ok = true;
            auto keys_times = [&](unsigned i) {     // step i's scores
                const unsigned g = i & 1, n = base + 2 * (PAIR ? i >> 1 : i), slot = n % ST;
                if (!(ok = bar_wait(full + 8 * slot, n / ST & 1, dead))) return;
                fence_after();
                const unsigned qa = q_at + (PAIR ? g * TILE : 0), ka = smem_u32(smem + slot * TILE);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    if (k < (int)ksteps)
                        multiply(tmem + 128 * g, operand(qa + (k >> 2) * KT * 128 + (k & 3) * 32, 0),
                                 operand(ka + (k >> 2) * KT * 128 + (k & 3) * 32, 0), product<T>(KT, false), k > 0);
                commit(s_full + 8 * g);
                if (!PAIR || g == 1) commit(empty + 8 * slot);
            };
            while (ok && w.next(a)) {
                if (row0 >= (unsigned)w.s.count * group) continue;
                const unsigned tiles = w.tile1 - w.tile0, steps = PAIR ? 2 * tiles : tiles;
                if (!(ok = bar_wait(q_ready, stretch & 1, dead))) break;
                fence_after();
                keys_times(0);
                if (ok && steps > 1) keys_times(1);
                for (unsigned i = 0; ok && i < steps; ++i) {
                    const unsigned g = i & 1, n = base + 2 * (PAIR ? i >> 1 : i) + 1, slot = n % ST;
                    if (!(ok = bar_wait(p_ready + 8 * g, ready[g] & 1, dead))) break;
                    ++ready[g];
                    if (!(ok = bar_wait(full + 8 * slot, n / ST & 1, dead))) break;
                    fence_after();
                    const unsigned va = smem_u32(smem + slot * TILE);
#pragma unroll
                    for (int k = 0; k < KT / 16; ++k)   // 16 keys: two groups of 8 rows
                        multiply_t(tmem + 256 + 128 * g, tmem + 128 * g + k * 8, operand(va + k * 2048, KT * 128), product<T>(DP, true),
                                   i > 1 || k > 0);
                    if (!PAIR || g == 1) commit(empty + 8 * slot);
                    if (i + 2 < steps) keys_times(i + 2);
                    else commit(o_full + 8 * g);
                }
                base += 2 * tiles;
                ++stretch;
            }
        }
        __syncwarp();
    } else {                   // the softmax: a thread a row
        const unsigned g = warp >> 2, r = t & 127u, lanes = (warp & 3u) << 21;   // this warp's lanes of tensor memory
        const unsigned my_s = tmem + 128 * g + lanes, my_o = tmem + 256 + 128 * g + lanes;
        const unsigned my_row = row0 + (PAIR ? g * 128 : 0) + r;
        const unsigned slot_floats = M * (dim + 2);
        float *slots = a.work + (size_t)gridDim.x * kRecord + (size_t)cta * 2 * slot_floats;
        unsigned phase = 0;    // steps of this group
        unsigned outs = 0;     // phases of o_full
        Meeting meet{smem_u32(&tail.meet), 0};
        bool ok = true;
        while (ok && w.next(a)) {
            const Span &s = w.s;
            const unsigned b = w.b, h = w.h, live = (unsigned)s.count * group;
            if (w.tile0 == 0 && s.bad && rt == 0 && h == 0 && t == 0 && a.c.status) atomicOr(a.c.status, PER_DEVFLAG_BAD_INDEX);
            if (w.tile0 == 0) absent_rows<T>(a, by_group, b, h, live, row0, M, t, kGroups * 128);
            if (w.tile0 == 0 && w.tile1 < w.n_tiles && t == 0) w.note(record, team);
            if (row0 >= live) continue;
            {                  // the queries, zero where there is none
                // eight requests at a time, so that their latencies overlap
                constexpr unsigned CH = DP / 8, ALL = M * CH / (kGroups * 128), EACH = ALL < 8 ? ALL : 8;
                const T *q = static_cast<const T *>(a.q) + b * a.sq[0];
#pragma unroll 1
                for (unsigned u0 = 0; u0 < ALL; u0 += EACH) {
                    uint4 v[EACH];
#pragma unroll
                    for (unsigned i = 0; i < EACH; ++i) {
                        const unsigned u = t + (u0 + i) * kGroups * 128, x = u / CH, c = u % CH;
                        const bool some = row0 + x < live;
                        const unsigned node = by_group.div(row0 + x), head = h * group + row0 + x - node * group;
                        const T *src = some ? q + node * a.sq[1] + head * a.sq[2] : q;
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (!a.qvec) v[i] = entries<T>(src, c, dim, some);
                        else if (some && c * 8 < dim) v[i] = *reinterpret_cast<const uint4 *>(src + c * 8);
                    }
#pragma unroll
                    for (unsigned i = 0; i < EACH; ++i) {
                        const unsigned u = t + (u0 + i) * kGroups * 128, x = u / CH, c = u % CH;
                        *reinterpret_cast<uint4 *>(qs + (x >> 7) * TILE + piece(KT, x & 127u, c)) = v[i];
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(q_ready);
            }
            const int node = my_row < live ? (int)by_group.div(my_row) : -1;
            const unsigned tiles = w.tile1 - w.tile0;
            float top = -INFINITY, l = 0.0f;      // what p refers to (in log2; -inf: nothing seen yet), and the sum of p
            float taken = 0.0f;                   // what is taken off the row's scores
            // before there is anything to wait for: whether the stretch has a page that does not exist (then, and at the
            // sequence's end, a tile's values are waited for before its scores are used), and what the row sees of the
            // first tile with nodes
            bool holes = false;
            {
                const unsigned last = min(w.tile1 * KT, (unsigned)s.total);
                if (w.tile0 * KT < last)
                    for (unsigned pg = a.c.page.div(w.tile0 * KT) + lane, end = a.c.page.div(last - 1); pg <= end; pg += 32)
                        holes |= (unsigned)a.c.table[b * a.c.st + pg] >= a.c.pages;
                holes = __any_sync(0xffffffffu, holes);
            }
            unsigned word[KT / 32] = {}, known = (unsigned)s.len / KT;
            if (known >= w.tile0 && known < w.tile1 && (PAIR || (known - w.tile0 & 1u) == g))
                seen(a, b, s, node, known * KT, nullptr, false, shift, word);
            for (unsigned j = PAIR ? 0 : g; j < tiles; j += PAIR ? 1 : 2) {
                const unsigned tile = w.tile0 + j, n = base + 2 * j + 1, slot = n % ST;
                const bool tail_in = (tile + 1) * KT > (unsigned)s.len;   // nodes, or the end
                ok = bar_wait(s_full + 8 * g, phase & 1, dead);
                if (ok && (tail_in || holes)) ok = bar_wait(full + 8 * slot, n / ST & 1, dead);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                ++phase;
                fence_after();
                if (tail_in && (!PAIR || g == 0)) {
                    // what stale slots hold is taken out of the values, and what is not finite in a node's: it must
                    // reach only the rows that see it
                    if (clean<T>(smem + slot * TILE, KT, tile * KT, s, halves * 8, r, 128)) tail.odd = 1;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                const bool masked = tail_in || holes;
                if (masked) {
                    if (tile != known || holes) {
                        seen(a, b, s, node, tile * KT, tail.bad[slot], holes, shift, word);
                        known = ~0u;
                    }
                    if (__any_sync(0xffffffffu, taken != 0.0f)) take_off(my_s, taken);
                }
                // p against the maximum so far, a quarter of the row at a time, and the row's maximum on the way; once more
                // where that has risen (the scores are still there: p is written when it stands)
                unsigned p[KT / 2];
                F2 add[2];
                for (;;) {
                    const float off = top == -INFINITY ? 0.0f : top - kUp<T>;
                    const F2 c2 = {a.c2, a.c2}, less = {-off, -off};
                    float most = -INFINITY;
                    add[0] = add[1] = F2{0.0f, 0.0f};
                    float two[2][32];         // a quarter that is worked on, and the next one on its way
                    get32(two[0], my_s);
#pragma unroll
                    for (int i = 0; i < KT / 32; ++i) {
                        float *sc = two[i & 1];
                        wait_ld();
                        loaded32(sc);
                        if (i + 1 < KT / 32) get32(two[(i + 1) & 1], my_s + 32 * (i + 1));
                        if (masked) hide(sc, word[i]);
                        float up[4] = {most, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int k = 0; k < 32; k += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e) up[e] = fmaxf(up[e], fmaxf(sc[k + e], sc[k + 4 + e]));
                        most = fmaxf(fmaxf(up[0], up[1]), fmaxf(up[2], up[3]));
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            F2 x = fma2(F2{sc[2 * k], sc[2 * k + 1]}, c2, less);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            add[k & 1] = add[k & 1] + x;
                            p[16 * i + k] = pack2<T>(x.x, x.y);
                        }
                    }
                    // (NaN, no rise, where nothing is seen even now)
                    const bool rise = fmaf(most, a.c2, -top) > kRise<T>;
                    if (!__any_sync(0xffffffffu, rise)) break;
                    const float now = most * a.c2;
                    float keep = rise ? ex2(top - now) : 1.0f;
                    const bool far = rise && !(fabsf(now) < kFar);
                    if (__any_sync(0xffffffffu, far)) {
                        holes = true;             // (the tiles to come take the way with the branches)
                        take_off(my_s, far ? most : 0.0f);
                        if (far) {
                            keep = ex2(fmaf(-most, a.c2, top));
                            taken += most;
                        }
                    }
                    if (rise) top = far ? 0.0f : now;
                    l *= keep;
                    if (j >= 2 || (PAIR && j >= 1)) {   // there are outputs
#pragma unroll 1
                        for (int i = 0; i < DP / 32; ++i) {
                            float x[32];
                            get32(x, my_o + 32 * i);
                            wait_ld();
                            loaded32(x);
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] *= keep;
                            put32(my_o + 32 * i, x);
                        }
                    }
                }
                put32(my_s, p);
                put32(my_s + 32, p + 32);
                l += (add[0].x + add[1].x) + (add[0].y + add[1].y);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(p_ready + 8 * g);
            }
            if (!ok) break;
            const bool has = PAIR || g < tiles;
            if (has) ok = __all_sync(0xffffffffu, bar_wait(o_full + 8 * g, outs & 1, dead));
            if (!ok) break;
            if (has) ++outs;
            const float mine = fmaf(taken, a.c2, top) - kUp<T>;
            if constexpr (!PAIR) {
                tail.ml[g * 128 + r][0] = mine;
                tail.ml[g * 128 + r][1] = l;
            }
            if (!(ok = meet(dead))) break;
            fence_after();
            const bool odd = *(volatile unsigned *)&tail.odd != 0;

            // a group's rows, or (of rows that both have) half of the entries
            const RowOut<T> out{a, by_group, b, h, live, row0, (unsigned)M, w.part(), slots + (w.tile0 != 0 ? 0 : slot_floats)};
            const unsigned row_in = (PAIR ? g * 128 : 0) + r;
            float f0 = 1.0f, f1 = 0.0f, m = mine, sum = l;
            const bool both = !PAIR && tiles > 1;
            if constexpr (!PAIR) {
                m = tail.ml[r][0];
                sum = tail.ml[r][1];
                if (both) {
                    const float m1 = tail.ml[128 + r][0], up = fmaxf(m, m1), least = up == -INFINITY ? 0.0f : up;
                    f0 = ex2(m - least);
                    f1 = ex2(m1 - least);
                    sum = sum * f0 + tail.ml[128 + r][1] * f1;
                    m = up;
                }
            }
            const unsigned o_at = PAIR ? my_o : tmem + 256 + lanes;
            const bool real = my_row < live;
            constexpr int HALF = DP / 32 / (PAIR ? 1 : 2);                // blocks of 32 entries a thread takes
#pragma unroll 1
            for (int i = 0; i < HALF; ++i) {
                const int c = (PAIR ? 0 : g * HALF) + i;
                float o[32];
                get32(o, o_at + 32 * c);
                if (both) {
                    float y[32];
                    get32(y, o_at + 128 + 32 * c);
                    wait_ld();
                    loaded32(o);
                    loaded32(y);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = o[k] * f0 + y[k] * f1;
                } else {
                    wait_ld();
                    loaded32(o);
                }
                if (odd && real) {   // what was taken out of the values, for the rows that see it (rare: nothing here is fast)
                    const unsigned first = max(w.tile0 * KT, (unsigned)s.len), end = min(w.tile1 * KT, (unsigned)s.total);
                    for (unsigned key = first; key < end; ++key) {
                        const unsigned pg = a.c.page.div(key);
                        const int e = a.c.table[b * a.c.st + pg];
                        if ((unsigned)e >= a.c.pages || !sees(a, b, s, node, key)) continue;
                        const T *src = static_cast<const T *>(a.c.v) + e * a.c.sv[0] + (key - pg * a.c.page.d) * a.c.sv[1] + h * a.c.sv[2];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float z = c * 32 + k < (int)dim ? to_f32(src[c * 32 + k]) : 0.0f;
                            if (!finite(z)) o[k] += z;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) out.put8(row_in, c * 32 + k * 8, o + 8 * k, m, sum);
            }
            fence_before();
            if (!(ok = meet(dead))) break;   // outputs, sums and the flag are read
            if (t == 0) tail.odd = 0;
            base += 2 * tiles;
        }
    }
    fence_before();
    __syncthreads();
    if (tail.dead[0]) {          // a wait gave up, be it the last one: nobody leaves, and tensor memory stays, before the copies
        if (t == 0 && a.c.status) atomicOr(a.c.status, PER_DEVFLAG_TIMEOUT);   // and products under way are done
        if (warp == 9 && chosen()) {   // the thread that issued them
            unsigned none[2] = {0, a.wait_ms};
            commit(smem_u32(&tail.last));
            bar_wait(smem_u32(&tail.last), 0, none);
        }
        __syncwarp();
        if (warp == 8 || warp == 10) {
            const unsigned val = warp == 10, asked = tail.asked[val];
            for (unsigned i = asked > (unsigned)ST + 1 ? asked - (ST + 1) / 2 * 2 : val; i < asked; i += 2) {
                unsigned none[2] = {0, a.wait_ms};
                bar_wait(full + 8 * (i % ST), i / ST & 1, none);
            }
        }
        __syncthreads();
    }
    if (warp == 9) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kColumns));
    }
}

template <typename T, int DP, bool PAIR>
cudaError_t wide(AttendArgs a, int type, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    using C = Cfg<DP, PAIR>;
    const Plan p = plan_of(a, C::M, KT, (unsigned)dev.sms, kBegin, false, false);
    if (bytes) {
        *bytes = p.parts ? p.bytes : 0;
        return cudaSuccess;
    }
    CacheMaps maps;
    unsigned shift;
    if (!make_maps(type, a, KT, &maps, &shift)) return cudaErrorInvalidValue;
    static std::atomic<bool> done[64];   // (two threads may both set the attribute, to the same value)
    if (!done[dev.device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(k_attend_wide<T, DP, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        done[dev.device].store(true, std::memory_order_release);
    }
    if (!p.parts) a.work = nullptr;
    FastDiv by_group;
    by_group.set(a.q_heads / a.c.heads);
    const cudaError_t e = launch_clusters(k_attend_wide<T, DP, PAIR>, p.grid, kThreads, 1, C::SMEM, st, maps, a, p.row_tiles, p.teams,
                                          by_group, shift);
    return e != cudaSuccess || !p.parts ? e : join_parts(type, a, p, by_group, st);
}

template <typename T>
cudaError_t wide_t(const AttendArgs &a, int type, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    const bool pair = a.nodes * (a.q_heads / a.c.heads) > 128;
    if (a.c.dim <= 64)
        return pair ? wide<T, 64, true>(a, type, dev, st, bytes) : wide<T, 64, false>(a, type, dev, st, bytes);
    return pair ? wide<T, 128, true>(a, type, dev, st, bytes) : wide<T, 128, false>(a, type, dev, st, bytes);
}

}  // namespace

cudaError_t attend_wide(int type, const AttendArgs &a, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    if (type == PER_TYPE_F16) return wide_t<__half>(a, type, dev, st, bytes);
    return wide_t<__nv_bfloat16>(a, type, dev, st, bytes);
}

}  // namespace attend
}  // namespace gbper
