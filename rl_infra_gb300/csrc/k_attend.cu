// k_attend.cu -- attention of drafted trees over a paged cache: which kernel takes a call, the one for layouts
// that the copy engine does not take, and the one that joins parts.
//
// Mathematics.  A pass over the keys with the running maximum m and sum l of a softmax: for each tile,
// s = scale q k, m' = max(m, max s), p = 2^(s - m'), l = l 2^(m - m') + sum p, o = o 2^(m - m') + p v (scores in units of
// log2).  Parts of a sequence join the same way.  Scores, sums and outputs are binary32; p is rounded
// to the type of v for the matrix instruction, whose products are exact (where few rows share a head of keys, taken in two
// parts: `values` in attend_mma.cuh).  binary32 operands are split into two parts of
// 11 bits, and the product of the two lower parts is dropped.
//
// The kernel here takes any strides and alignment: 64 rows a CTA, 16 a warp, entries copied one by one.
#include "attend_mma.cuh"

#include <algorithm>
#include <atomic>

namespace gbper {
namespace attend {
namespace {

constexpr int kThreads = 128;
constexpr unsigned kBegin = 2;   // tiles that a sequence's begin and end are worth
// Rows of a head of keys that the warp-wide instruction takes: it is quicker to begin, the tensor cores' own one to go on
// (16 trees, up to 4000 tokens: 48 rows 64.6 us against 79.7 warp-wide; 16 of 8000, 32 rows 83 us warp-wide against 108).
constexpr unsigned kFew = 32;

template <typename T, int DP>
struct Cfg {
    static constexpr int ES = (int)sizeof(T);
    static constexpr int KT = DP * ES > 512 ? 32 : 64;      // keys of a tile
    static constexpr int M = 64;                            // rows of a CTA
    static constexpr int CH = DP * ES / 16;                 // pieces of a row
    static constexpr int TILE = KT * DP * ES;
    static constexpr int QB = M * DP * ES * (ES == 4 ? 2 : 1);   // binary32: both parts of each
    static constexpr int SMEM = 2 * TILE + QB + KT * 16 + 64;
    static_assert(KT * 16 >= M * 8 && DP * ES >= 64, "what goes out fits where queries and places were");
    static constexpr int PER_SM = 227 * 1024 / (SMEM + 1024) < 3 ? 227 * 1024 / (SMEM + 1024) : 3;
};

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) k_attend_any(AttendArgs a, unsigned row_tiles, unsigned max_teams, FastDiv by_group)
{
    using C = Cfg<T, DP>;
    constexpr int KT = C::KT, M = C::M, ES = C::ES;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *ks = smem, *vs = smem + C::TILE, *qs = smem + 2 * C::TILE;
    longlong2 *info = reinterpret_cast<longlong2 *>(qs + C::QB);   // [KT] element offsets of keys and values
    unsigned *valid = reinterpret_cast<unsigned *>(info + KT);           // [2] bits: the key is there
    u64 *scan = reinterpret_cast<u64 *>(valid + 2);                      // [4]
    const unsigned t = threadIdx.x, lane = t & 31u, warp = t >> 5;
    const unsigned g = lane >> 2, q4 = lane & 3u;                  // row and column pair of a fragment
    const unsigned cta = blockIdx.x, team = cta / row_tiles, rt = cta - team * row_tiles;
    const unsigned group = by_group.d, row0 = rt * M, dim = a.c.dim;
    const unsigned halves = (dim * ES + 127) / 128;
    const unsigned slot_floats = M * (dim + 2);
    int *record = reinterpret_cast<int *>(a.work) + (size_t)cta * kRecord;
    float *slots = a.work + (size_t)gridDim.x * kRecord + (size_t)cta * 2 * slot_floats;

    pdl_wait();
    pdl_release();
    if (a.work && t == 0) record[3] = 0;
    Walk<KT, kBegin> w;
    if (!w.template begin<kThreads>(a, team, max_teams, scan)) return;
    while (w.next(a)) {
        const Span &s = w.s;
        const unsigned b = w.b, h = w.h;
        if (w.tile0 == 0 && s.bad && rt == 0 && h == 0 && t == 0 && a.c.status) atomicOr(a.c.status, PER_DEVFLAG_BAD_INDEX);
        const unsigned live = (unsigned)s.count * group;          // rows of nodes that are there
        if (w.tile0 == 0) absent_rows<T>(a, by_group, b, h, live, row0, M, t, kThreads);
        if (w.tile0 == 0 && w.tile1 < w.n_tiles && t == 0) w.note(record, team);
        if (row0 >= live) continue;

        // the queries, zero where there is none
        __syncthreads();
        {
            const T *q = static_cast<const T *>(a.q) + b * a.sq[0];
            for (unsigned u = t; u < M * C::CH; u += kThreads) {
                const unsigned r = u / C::CH, c = u % C::CH;
                const bool some = row0 + r < live;
                const unsigned node = by_group.div(row0 + r), head = h * group + row0 + r - node * group;
                const T *src = some ? q + node * a.sq[1] + head * a.sq[2] : q;
                uint4 v = entries<T>(src, c, dim, some);
                if constexpr (ES == 4) {
                    uint4 lo;
                    split(__uint_as_float(v.x), v.x, lo.x);
                    split(__uint_as_float(v.y), v.y, lo.y);
                    split(__uint_as_float(v.z), v.z, lo.z);
                    split(__uint_as_float(v.w), v.w, lo.w);
                    *reinterpret_cast<uint4 *>(qs + M * DP * ES + piece(M, r, c)) = lo;
                }
                *reinterpret_cast<uint4 *>(qs + piece(M, r, c)) = v;
            }
        }
        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
        int node[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const unsigned r = row0 + warp * 16 + g + e * 8;
            node[e] = r < live ? (int)by_group.div(r) : -1;       // -1: no such row
        }
        for (unsigned tile = w.tile0; tile < w.tile1; ++tile) {
            __syncthreads();                                      // the tile before is done with
            if (t < KT) {                                         // where its keys lie
                const unsigned key = tile * KT + t;
                longlong2 x = make_longlong2(0, 0);
                bool there = key < (unsigned)s.total;
                if (there) {
                    const unsigned pg = a.c.page.div(key), slot = key - pg * a.c.page.d;
                    const int e = a.c.table[b * a.c.st + pg];
                    there = e >= 0 && (unsigned)e < a.c.pages;
                    if (there) {
                        x.x = e * a.c.sk[0] + slot * a.c.sk[1] + h * a.c.sk[2];
                        x.y = e * a.c.sv[0] + slot * a.c.sv[1] + h * a.c.sv[2];
                    } else if (rt == 0 && h == 0 && a.c.status) {
                        atomicOr(a.c.status, PER_DEVFLAG_BAD_INDEX);
                    }
                }
                const unsigned bits = __ballot_sync(0xffffffffu, there);
                if (lane == 0) valid[warp] = bits;
                info[t] = x;
            }
            __syncthreads();
            const unsigned there0 = valid[0], there1 = KT > 32 ? valid[1] : ~0u;
            for (unsigned u = t; u < KT * C::CH; u += kThreads) {
                const unsigned r = u / C::CH, c = u % C::CH;
                const bool some = (r < 32 ? there0 : there1) >> (r & 31u) & 1u;
                const longlong2 x = info[r];
                *reinterpret_cast<uint4 *>(ks + piece(KT, r, c)) = entries<T>(static_cast<const T *>(a.c.k) + x.x, c, dim, some);
                *reinterpret_cast<uint4 *>(vs + piece(KT, r, c)) = entries<T>(static_cast<const T *>(a.c.v) + x.y, c, dim, some);
            }
            __syncthreads();
            const bool nodes_in = (tile + 1) * KT > (unsigned)s.len;
            const bool masked = nodes_in || (there0 & there1) != ~0u;

            // a value that is not finite must reach only the rows that see it
            bool odd = false;
            if (nodes_in) {
                for (unsigned u = t; u < KT * C::CH; u += kThreads)
                    if (tile * KT + u / C::CH >= (unsigned)s.len)
                        odd |= take_out<T>(reinterpret_cast<uint4 *>(vs + piece(KT, u / C::CH, u % C::CH)));
                odd = __syncthreads_or(odd);
            }

            float sc[KT / 8][4];
            scores<T, DP, KT>(sc, qs, M, warp * 16, ks, KT, 0, halves);
#pragma unroll
            for (int i = 0; i < KT / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[i][e] *= a.c2;
            if (masked)
                hide<KT>(sc, a, b, s, node, tile * KT, 0, [&](unsigned r) { return ((r < 32 ? there0 : there1) >> (r & 31u) & 1u) != 0; });
            if constexpr (ES == 4) once_more<KT>(sc, a, b, h, group, node, row0 + warp * 16 + g, ks, KT, 0);
            soften<T, DP, KT>(sc, top, sum, o);
            values<T, DP, KT, false>(o, sc, vs, KT, 0, halves);
            if (odd)
                for (unsigned r = 0; r < KT; ++r) {
                    const unsigned key = tile * KT + r;
                    if ((int)key < s.len || !(((r < 32 ? there0 : there1) >> (r & 31u)) & 1u)) continue;
                    give_back<T, DP>(a, b, s, node, key, static_cast<const T *>(a.c.v) + info[r].y, o);
                }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
            sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
            top[e] = below<T>(top[e]);      // from here on what the sums refer to
        }
        // out, by way of the queries' place, 16 columns at a time
        const RowOut<T> out{a, by_group, b, h, live, row0, M, w.part(), slots + (w.tile0 != 0 ? 0 : slot_floats)};
        float *sums = reinterpret_cast<float *>(qs);                  // [M][16]
        float *ml = reinterpret_cast<float *>(info);                  // [M][2]
#pragma unroll
        for (int d0 = 0; d0 < DP; d0 += 16) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const unsigned r = warp * 16 + g + e * 8;
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    *reinterpret_cast<float2 *>(sums + r * 16 + k * 8 + q4 * 2) = make_float2(o[d0 / 8 + k][2 * e], o[d0 / 8 + k][2 * e + 1]);
                if (q4 == 0) {
                    ml[2 * r] = top[e];
                    ml[2 * r + 1] = sum[e];
                }
            }
            __syncthreads();
            const unsigned r = t / 2, c = t % 2 * 8;                  // 128 threads, 64 rows of two eights
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = sums[r * 16 + c + e];
            out.put8(r, d0 + c, x, ml[2 * r], ml[2 * r + 1]);
        }
    }
}

// Joins the parts of what lies in several CTAs: each CTA that begins such a stretch left a record.  LR lanes take a row,
// eight entries each; they work out the weights of LR parts at once.
template <typename T, int LR>
__global__ void __launch_bounds__(kThreads) k_attend_join(AttendArgs a, unsigned row_tiles, unsigned m_rows, FastDiv by_group)
{
    const unsigned cta = blockIdx.x, team = cta / row_tiles, rt = cta - team * row_tiles;
    pdl_wait();
    pdl_release();
    const int4 record = *(reinterpret_cast<const int4 *>(a.work) + (size_t)cta * (kRecord / 4));
    const int parts = record.w;
    if (parts == 0) return;
    const unsigned b = (unsigned)record.x, h = (unsigned)record.y, count = (unsigned)record.z;
    const unsigned live = count * by_group.d, dim = a.c.dim, slot_floats = m_rows * (dim + 2);
    const unsigned lane = threadIdx.x & 31u, li = lane & (LR - 1);
    const unsigned r = blockIdx.y * (kThreads / LR) + threadIdx.x / LR;
    const bool real = r < m_rows && rt * m_rows + r < live;
    if (!__any_sync(0xffffffffu, real)) return;
    const unsigned row = real ? r : 0;
    const float *slots = a.work + (size_t)gridDim.x * kRecord;
    auto slot = [&](int i) {   // the first part lies in its CTA's second slot, the others in their first
        return slots + ((size_t)((team + i) * row_tiles + rt) * 2 + (i == 0)) * slot_floats;
    };
    float m = -INFINITY;
    for (int i = li; i < parts; i += LR) m = fmaxf(m, slot(i)[m_rows * dim + 2 * row]);
#pragma unroll
    for (int d = LR / 2; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float base = m == -INFINITY ? 0.0f : m;
    float x[8] = {}, l = 0.0f;
    for (int i0 = 0; i0 < parts; i0 += LR) {
        float f = 0.0f;
        if (i0 + (int)li < parts) {
            const float2 z = *reinterpret_cast<const float2 *>(slot(i0 + li) + m_rows * dim + 2 * row);
            f = ex2(z.x - base);
            l += f * z.y;
        }
        const int n = min(LR, parts - i0);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float w = __shfl_sync(0xffffffffu, f, i, LR);
            const float *p = slot(i0 + i) + row * dim + li * 8;
            if (li * 8 >= dim) continue;
            if (dim % 8 == 0) {
                const float4 y = *reinterpret_cast<const float4 *>(p), z = *reinterpret_cast<const float4 *>(p + 4);
                x[0] += w * y.x, x[1] += w * y.y, x[2] += w * y.z, x[3] += w * y.w;
                x[4] += w * z.x, x[5] += w * z.y, x[6] += w * z.z, x[7] += w * z.w;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (li * 8 + e < dim) x[e] += w * p[e];
            }
        }
    }
#pragma unroll
    for (int d = LR / 2; d; d /= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
    const RowOut<T> out{a, by_group, b, h, live, rt * m_rows, m_rows, false, nullptr};
    if (real) out.put8(r, li * 8, x, m, l);
}

// ---- the copy engine's maps ----------------------------------------------------------------------
typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                           const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                           CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder()
{
    static std::atomic<void *> known{nullptr};
    void *f = known.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        known.store(f, std::memory_order_release);
    }
    return reinterpret_cast<Encode>(f);
}

// One array as the copy engine sees it, its axes in the order of their strides.  False: it does not take it (each stride
// must be a multiple of the one before and past all that this covers).
struct Layout {
    cuuint64_t size[4], stride[3];
    int slot_axis;
    unsigned char at[3];
};

bool layout_of(const AttendArgs &a, const long long st[3], unsigned es, Layout *l)
{
    const u64 dims[3] = {a.c.page.d, a.c.heads, a.c.pages};   // slot, head, page
    const long long strides[3] = {st[1], st[2], st[0]};
    int order[3] = {0, 1, 2};
    auto before = [&](int x, int y) {
        if ((dims[x] == 1) != (dims[y] == 1)) return dims[y] == 1;   // axes of one place last
        return dims[x] == 1 || strides[x] == strides[y] ? x < y : strides[x] < strides[y];
    };
    if (before(order[1], order[0])) std::swap(order[0], order[1]);
    if (before(order[2], order[1])) std::swap(order[1], order[2]);
    if (before(order[1], order[0])) std::swap(order[0], order[1]);
    l->size[0] = a.c.dim;
    u64 unit = 16, covered = (u64)a.c.dim * es;
    for (int i = 0; i < 3; ++i) {
        const int x = order[i];
        u64 s = (covered + unit - 1) / unit * unit;            // an axis of one place: any stride would do
        if (dims[x] > 1) {
            if (strides[x] <= 0) return false;
            s = (u64)strides[x] * es;
            if (s < covered || s % unit) return false;
        }
        if (s >= 1ull << 40) return false;
        l->size[i + 1] = dims[x];
        l->stride[i] = s;
        if (x == 0) l->slot_axis = i + 1;
        l->at[x] = (unsigned char)(i + 1);
        covered += s * (dims[x] - 1);
        unit = s;
    }
    return true;
}

bool make_map(int type, const AttendArgs &a, const void *base, const long long st[3], unsigned rows, CUtensorMap *map, unsigned char *at)
{
    const Encode encode = encoder();
    const unsigned es = type == PER_TYPE_F32 ? 4 : 2;
    Layout l;
    if (!encode || !layout_of(a, st, es, &l)) return false;
    cuuint32_t box[4] = {128 / es, 1, 1, 1}, one[4] = {1, 1, 1, 1};
    box[l.slot_axis] = rows;
    for (int i = 0; i < 3; ++i) at[i] = l.at[i];
    const CUtensorMapDataType kind = type == PER_TYPE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : type == PER_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode(map, kind, 4, const_cast<void *>(base), l.size, l.stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DP>
cudaError_t attend_any(AttendArgs a, int type, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    using C = Cfg<T, DP>;
    const Plan p = plan_of(a, C::M, C::KT, (unsigned)dev.sms * C::PER_SM, kBegin, false, false);
    if (bytes) {
        *bytes = p.parts ? p.bytes : 0;
        return cudaSuccess;
    }
    static std::atomic<bool> done[64];   // (two threads may both set the attribute, to the same value)
    if (!done[dev.device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(k_attend_any<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        done[dev.device].store(true, std::memory_order_release);
    }
    if (!p.parts) a.work = nullptr;
    FastDiv by_group;
    by_group.set(a.q_heads / a.c.heads);
    const cudaError_t e = launch_clusters(k_attend_any<T, DP>, p.grid, kThreads, 1, C::SMEM, st, a, p.row_tiles, p.teams, by_group);
    return e != cudaSuccess || !p.parts ? e : join_parts(type, a, p, by_group, st);
}

template <typename T>
cudaError_t attend_any_t(const AttendArgs &a, int type, const DeviceInfo &dev, cudaStream_t st, u64 *bytes)
{
    if (a.c.dim <= 64) return attend_any<T, 64>(a, type, dev, st, bytes);
    if (a.c.dim <= 128) return attend_any<T, 128>(a, type, dev, st, bytes);
    return attend_any<T, 256>(a, type, dev, st, bytes);
}

// Launches, or (bytes given) says what scratch memory the call needs.
cudaError_t attend(int type, const AttendArgs &a, cudaStream_t st, u64 *bytes)
{
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    if (bytes) *bytes = 0;
    const unsigned es = type == PER_TYPE_F32 ? 4 : 2;
    Layout l;
    if (a.c.vec && a.c.pages && a.c.width && encoder() && layout_of(a, a.c.sk, es, &l) && layout_of(a, a.c.sv, es, &l)) {
        if (type == PER_TYPE_F32) return attend_rows_f32(a, dev, st, bytes);
        if (a.c.dim <= 128 && a.nodes * (a.q_heads / a.c.heads) > kFew && a.c2 > 0.0f) return attend_wide(type, a, dev, st, bytes);
        return type == PER_TYPE_F16 ? attend_rows_f16(a, dev, st, bytes) : attend_rows_bf16(a, dev, st, bytes);
    }
    if (type == PER_TYPE_F32) return attend_any_t<float>(a, type, dev, st, bytes);
    if (type == PER_TYPE_F16) return attend_any_t<__half>(a, type, dev, st, bytes);
    return attend_any_t<__nv_bfloat16>(a, type, dev, st, bytes);
}

}  // namespace

bool make_maps(int type, const AttendArgs &a, unsigned kt, CacheMaps *maps, unsigned *shift)
{
    unsigned s = 0;                // rows of a box: a power of 2 that divides the page
    while ((2u << s) <= kt && a.c.page.d % (2u << s) == 0) ++s;
    *shift = s;
    return make_map(type, a, a.c.k, a.c.sk, 1u << s, &maps->k, maps->k_at) && make_map(type, a, a.c.v, a.c.sv, 1u << s, &maps->v, maps->v_at);
}

namespace {

template <typename T, int LR>
cudaError_t join(const AttendArgs &a, const Plan &p, const FastDiv &by_group, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid, (p.m + kThreads / LR - 1) / (kThreads / LR));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attend_join<T, LR>, a, p.row_tiles, p.m, by_group);
}

template <typename T>
cudaError_t join_t(const AttendArgs &a, const Plan &p, const FastDiv &by_group, cudaStream_t st)
{
    if (a.c.dim <= 64) return join<T, 8>(a, p, by_group, st);
    if (a.c.dim <= 128) return join<T, 16>(a, p, by_group, st);
    return join<T, 32>(a, p, by_group, st);
}

}  // namespace

cudaError_t join_parts(int type, const AttendArgs &a, const Plan &p, const FastDiv &by_group, cudaStream_t st)
{
    if (type == PER_TYPE_F32) return join_t<float>(a, p, by_group, st);
    if (type == PER_TYPE_F16) return join_t<__half>(a, p, by_group, st);
    return join_t<__nv_bfloat16>(a, p, by_group, st);
}

}  // namespace attend

cudaError_t launch_attend(int type, const AttendArgs &a, cudaStream_t st) { return attend::attend(type, a, st, nullptr); }

cudaError_t attend_work(int type, const AttendArgs &a, unsigned long long *bytes)
{
    return attend::attend(type, a, nullptr, bytes);
}

}  // namespace gbper
