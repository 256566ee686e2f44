// Differential attention over a paged cache on the tensor cores
// (include/paged.h), for bf16 and fp16.
//
// New tokens are few and keys are many, so the keys take the 128 rows of a
// product and the queries its columns: S_m = K_m q_m^T is [128 keys, RT], RT
// the rows (queries x the heads that share a key head) of a tile, and the sums
// are O^T = V^T [P_0 | P_1], [Dv, 2 RT]. A tile of 16 rows so costs 16 columns
// of a product and not 128, and a thread, which has one key of a step, turns RT
// scores of a map into weights. Row maxima are then over threads; they are
// formed only when some weight would exceed 2^8 of its row's first best, which
// one vote of a map's 128 threads per step finds out.
//
// The keys of all tiles, in steps of 128, are cut into equal shares for one CTA
// per SM: a CTA's share is an end of one tile, some whole tiles, and the
// beginning of another. Whole tiles go to the output directly; pieces leave
// their sums, maxima and weights' sums in one of the CTA's two slots, and a
// second kernel joins them. The shares are made on the device, from lengths and
// counts, so a captured graph stays balanced while its sequences grow.
//
// Warps: groups of four for the weights of up to 32 rows of a map, one that loads
// by TMA (a box lies in one page: gcd(page size, 128) places), one that issues the
// products. Weights go through shared memory, rounded to the inputs' type; tiles
// of up to 32 rows, which memory bounds, carry what that took as a second operand.
#pragma once

#include <cfloat>

#include "dattn_tc.cuh"
#include "paged_internal.cuh"

namespace da {
namespace {

using namespace tc;

constexpr int kStep = 128;            // keys
constexpr float kSlack = 8.f;         // log2 of how far weights may exceed their first best
template <typename T> constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;  // log2 of that best

using tc::tmem_load;
using tc::tmem_store;

// Columns addr .. of the warp's 32 lanes.
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
                 "}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                   "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const float (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
                 "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
                 "};"
                 :
                 : "r"(addr),
                   "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
                   "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
                 : "memory");
}

// A stage is [V | K_0 | K_1]: with VP = 64 the product's second 64 rows, which
// nothing reads, are of K.
template <int DP, int VP, int RT> struct PgShared {
    static constexpr int C = RT < 32 ? RT : 32;          // rows of a group of warps
    static constexpr int groups = 2 * RT / C;            // map 0's, then map 1's
    static constexpr int threads = groups * 128 + 64;
    static constexpr int row = DP * 2;                   // bytes of a row of q or k
    static constexpr int q = RT * row, k = kStep * row;  // of one map
    static constexpr int vblock = kStep * 128;           // of 64 columns of V
    static constexpr int v = VP / 64 * vblock;
    static constexpr int stage = v + 2 * k;
    static constexpr bool rests = RT <= 32;              // weights carry what rounding took
    static constexpr int prow = RT == 16 ? 64 : 128;     // bytes of a key's row of weights
    static constexpr int p = kStep * 2 * RT * 2;         // of both maps' weights
    static constexpr int pbuf = p * (rests ? 2 : 1);
    static constexpr int qbufs = RT == 64 ? 1 : 2;
    static constexpr int pbufs = RT == 64 ? 2 : 1;
    static constexpr int fixed = qbufs * 2 * q + pbufs * pbuf;
    static constexpr int arrays = RT * 96 + 768;         // the kernel's static ones, at most
    static constexpr int room = 227 * 1024 - 1024 - kPgBias - arrays;  // 1024 for alignment
    static constexpr int fit = (room - fixed) / stage;
    static constexpr int stages = fit > 6 ? 6 : fit;
    static constexpr int at_stage = qbufs * 2 * q, at_p = at_stage + stages * stage, bytes = at_p + pbufs * pbuf;
    static_assert(stages >= 2 && bytes <= room, "shared memory");
};

// What passes a phase ahead has a barrier for even and one for odd steps; the
// others' next phase cannot end before everyone has seen the last one.
// empty[s]: the products with P of a step are done, and its stage is free.
struct PgBars {
    uint64_t q_full[2], q_empty[2];
    uint64_t full[6], empty[6];
    uint64_t s_full[2], p_full[2];
    uint32_t tmem, gave_up;
};

__device__ uint32_t g_paged_gave_up;

// A tile of a sequence's rows: rt-th of sequence b (all key heads have the same).
struct Tile {
    int b, l0, len, count, end, steps;  // first query, keys, queries, keys that some query sees, steps of them
};

__device__ __forceinline__ Tile tile_of(const PagedTcArgs &a, int e)
{
    Tile t;
    t.b = e / a.row_tiles;
    t.l0 = (e - t.b * a.row_tiles) * a.LP;
    t.len = dattn_length(a.d, t.b);
    t.count = paged_count(a.d, t.b);
    t.end = t.l0 < t.count ? t.len : 0;
    // Keys after the tile's last query end the walk where positions are indices.
    if (a.d.causal && !a.d.pos_q && !a.d.pos_k) t.end = min(t.end, max(t.len - t.count + min(t.l0 + a.LP, t.count), 0));
    t.steps = max((t.end + kStep - 1) / kStep, 1);
    return t;
}

// A CTA's walk over its share, segment by segment: `steps` of tile (e, n) from `first` on.
struct Walk {
    int64_t left;
    int e, n, first, steps;
    Tile t;

    __device__ __forceinline__ void open() { steps = static_cast<int>(min(static_cast<int64_t>(t.steps - first), left)); }
    __device__ __forceinline__ void start(const PagedTcArgs &a, int64_t share, int e_, int n_, int first_)
    {
        left = share;
        e = e_;
        n = n_;
        first = first_;
        if (left > 0) {
            t = tile_of(a, e);
            open();
        }
    }
    __device__ __forceinline__ void next(const PagedTcArgs &a)
    {
        left -= steps;
        first = 0;
        if (left <= 0) return;
        if (++n == a.d.Hkv) {
            n = 0;
            t = tile_of(a, ++e);
        }
        open();
    }
};

// Sums of N columns over the warp's lanes; lane i is left with columns
// i * N / 32 .. (N >= 32), or with column i / 2 (N = 16).
template <int N> __device__ __forceinline__ void fold(float (&v)[N], int lane, int o)
{
    if constexpr (N == 1) {
        for (; o; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    } else if (o) {
        float h[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float keep = lane & o ? v[i + N / 2] : v[i], send = lane & o ? v[i] : v[i + N / 2];
            h[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
        fold<N / 2>(h, lane, o >> 1);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) v[i] = h[i];
    }
}

// Whether any of the 128 threads of a group has `flag`.
__device__ __forceinline__ bool vote(int group, bool flag)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                 "bar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(flag)), "r"(1 + group)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_group(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
template <int THREADS> __device__ __forceinline__ void sync_groups() { asm volatile("bar.sync 7, %0;" ::"n"(THREADS) : "memory"); }

// Whether a phase has ended, without waiting; the same in all lanes of a warp.
// kIdle tests of nothing to do, some 100 ns each, end the wait (bar_wait).
constexpr uint32_t kIdle = 10u << 20;
__device__ __forceinline__ bool bar_test(uint64_t *bar, uint32_t parity, volatile uint32_t *gave_up)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return __all_sync(0xffffffffu, ok != 0 || *gave_up);
}

// Maximum over the warp, by the floats' order as integers.
__device__ __forceinline__ float warp_max(float v)
{
    int i = __float_as_int(v);
    i = i >= 0 ? i : i ^ 0x7fffffff;
    i = __reduce_max_sync(0xffffffffu, i);
    return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff);
}

template <typename T, int DP, int VP, int RT>
__global__ void __launch_bounds__(PgShared<DP, VP, RT>::threads, 1)
    paged_tc_kernel(const __grid_constant__ PagedTcArgs a, const __grid_constant__ CUtensorMap mq,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv)
{
    using F = PgShared<DP, VP, RT>;
    constexpr int NS = F::stages, C = F::C, kThreads = F::threads, kLoad = F::groups * 4, kIssue = kLoad + 1;
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t columns = RT == 16 ? 128 : RT == 32 ? 256 : 512;
    extern __shared__ unsigned char raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    __shared__ PgBars bars;
    // Each group's rows.
    __shared__ __align__(16) float noff[F::groups][C];     // minus the row's reference
    __shared__ __align__(16) float shrink[F::groups][C];
    __shared__ __align__(16) float wide[F::groups][4][C];  // a warp's maxima, or sums
    __shared__ int row_pos[F::groups][C], row_l[F::groups][C], row_h[F::groups][C];
    __shared__ float far_bias[F::groups][2][C];            // of keys `reach` or more before and after the query
    __shared__ int64_t warp_total[kThreads / 32];
    __shared__ int start[3];
    float *table = reinterpret_cast<float *>(base + F::bytes);  // [nb][H], times log2(e)
    uint16_t *bmap = reinterpret_cast<uint16_t *>(table + a.d.nb * a.d.H);
    const DattnArgs &d = a.d;
    const int warp = warp_number(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            bar_init(&bars.q_full[i], 1);
            bar_init(&bars.q_empty[i], 1);
            bar_init(&bars.s_full[i], 1);
            bar_init(&bars.p_full[i], F::groups * 4);
        }
        for (int s = 0; s < NS; ++s) {
            bar_init(&bars.full[s], 1);
            bar_init(&bars.empty[s], 1);
        }
        bars.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
    }
    if (warp == kIssue) tmem_alloc(&bars.tmem, columns);
    for (int i = threadIdx.x; i < d.nb * d.H; i += kThreads) table[i] = d.table[i] * kLog2e;
    for (int i = threadIdx.x; i < 2 * d.reach + 1 && d.nb; i += kThreads)
        bmap[i] = static_cast<uint16_t>(min(max(d.bmap[i], 0), d.nb - 1) * d.H);
    // Rows of q that a tile's queries leave free.
    const int used = a.LP * d.G;
    for (int i = threadIdx.x; i < F::qbufs * 2 * (RT - used) * (F::row / 16); i += kThreads) {
        const int m = i / ((RT - used) * (F::row / 16)), rest = i - m * (RT - used) * (F::row / 16);
        *reinterpret_cast<uint4 *>(base + m * F::q + used * F::row + rest * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async();

    // The CTA's share: threads take consecutive tiles' steps, a scan adds them up.
    const int entries = d.B * a.row_tiles, per = (entries + kThreads - 1) / kThreads;
    const int e0 = min(static_cast<int>(threadIdx.x) * per, entries), e1 = min(e0 + per, entries);
    int64_t own = 0;
    for (int e = e0; e < e1; ++e) own += tile_of(a, e).steps;
    own *= d.Hkv;
    int64_t upto = own;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) warp_total[warp] = upto;
    fence_before();
    __syncthreads();
    fence_after();
    int64_t total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) upto += total;
        total += warp_total[w];
    }
    // CTAs without a share are the last ones, so that a tile's pieces lie in CTAs in a row.
    const int64_t active = min(total, static_cast<int64_t>(gridDim.x)), cta = min(static_cast<int64_t>(blockIdx.x), active);
    const int64_t from = total * cta / active, share = cta < active ? total * (cta + 1) / active - from : 0;
    if (share > 0 && from < upto && from >= upto - own) {
        int64_t at = upto - own;
        int e = e0, steps = 0;
        for (;; ++e) {
            steps = tile_of(a, e).steps;
            if (from < at + static_cast<int64_t>(steps) * d.Hkv) break;
            at += static_cast<int64_t>(steps) * d.Hkv;
        }
        start[0] = e;
        start[1] = static_cast<int>((from - at) / steps);
        start[2] = static_cast<int>((from - at) % steps);
    }
    __syncthreads();
    const uint32_t tmem = uniform(bars.tmem);
    volatile uint32_t *gave_up = &bars.gave_up;
    const auto tS = [&](int m, int t) { return tmem + ((t & 1) * 2 + m) * RT; };
    const uint32_t tO = tmem + 4 * RT;
    Walk w;
    w.start(a, share, start[0], start[1], start[2]);

    if (warp == kLoad) {
        const int boxes = kStep / a.box;  // of a step, one to a lane
        const int blocks = (d.Dv + 63) / 64;
        int t = 0, seg = 0;
        for (; w.left > 0; w.next(a), ++seg) {
            const int qb = seg % F::qbufs;
            bar_wait_warp(&bars.q_empty[qb], ((seg / F::qbufs) & 1) ^ 1, gave_up);
            if (lane == 0) {
                bar_expect(&bars.q_full[qb], 2 * F::row * used);
                for (int m = 0; m < 2; ++m) tma_load(&mq, &bars.q_full[qb], base + (qb * 2 + m) * F::q, 0, m, w.n * d.G, w.t.l0, w.t.b);
            }
            for (int i = 0; i < w.steps; ++i, ++t) {
                const int s = t % NS, j = (w.first + i) * kStep + lane * a.box;
                int place = 0, page = -1;
                if (lane < boxes && j < w.t.end) page = paged_page(d, w.t.b, j, place);
                const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
                bar_wait_warp(&bars.empty[s], ((t / NS) & 1) ^ 1, gave_up);
                if (lane == 0) bar_expect(&bars.full[s], __popc(there) * a.box * (2 * F::row + blocks * 128));
                __syncwarp();
                if (page >= 0) {
                    unsigned char *st = base + F::at_stage + s * F::stage;
                    for (int m = 0; m < 2; ++m) tma_load(&mk, &bars.full[s], st + F::v + m * F::k + lane * a.box * F::row, 0, m, w.n, place, page);
                    for (int c = 0; c < blocks; ++c) tma_load(&mv, &bars.full[s], st + c * F::vblock + lane * a.box * 128, c * 64, 0, w.n, place, page);
                }
                __syncwarp();
            }
        }
        if (*gave_up) {  // leave no copy in flight
            for (int i = max(0, seg - F::qbufs); i < seg; ++i) bar_drain(&bars.q_full[i % F::qbufs], (i / F::qbufs) & 1);
            for (int i = max(0, t - NS); i < t; ++i) bar_drain(&bars.full[i % NS], (i / NS) & 1);
        }
    } else if (warp == kIssue) {
        // All lanes walk through the steps, one issues: addresses then stay in
        // uniform registers.
        const bool issue = elect();
        constexpr uint32_t is = shape(bf16, RT, false), io = shape(bf16, 2 * RT, true) | (1u << 15);
        const uint32_t sb = smem_addr(base);
        const Operand<F::row> dk = along_row<F::row>(sb + F::at_stage + F::v), dq = along_row<F::row>(sb);
        const Operand<128> dv = over_rows<128>(sb + F::at_stage, F::vblock);
        const Operand<F::prow> dp = over_rows<F::prow>(sb + F::at_p, F::p / 2);
        // Scores of step u need its keys, and the weights of step u - 2 in
        // place of the scores that they overwrite; sums of step t need its
        // weights. Whichever can is issued next: sums that waited behind scores
        // would hold their stage for as long as the next keys take to arrive.
        Walk ws = w;
        const int steps = static_cast<int>(share);
        int u = 0, t = 0, at = 0, seg = 0, done = 0;  // scores and sums issued, scores of the segment, its number, sums of theirs
        for (uint32_t idle = 0; t < steps;) {
            const int qb = seg % F::qbufs;
            if (u < steps && u <= t + 1 && bar_test(&bars.full[u % NS], (u / NS) & 1, gave_up) &&
                (at > 0 || bar_test(&bars.q_full[qb], (seg / F::qbufs) & 1, gave_up))) {
                const int s = u % NS;
                const bool last = ++at == ws.steps;
                fence_after();
                if (issue) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i)
                            mma_ss(tS(m, u), dk.at(s * F::stage + m * F::k + i * 32), dq.at((qb * 2 + m) * F::q + i * 32), is, i > 0);
                    mma_commit(&bars.s_full[u & 1]);
                    if (last) mma_commit(&bars.q_empty[qb]);
                }
                __syncwarp();
                if (last) {
                    ws.next(a);
                    at = 0;
                    ++seg;
                }
                ++u;
                idle = 0;
            } else if (t < u && bar_test(&bars.p_full[t & 1], (t >> 1) & 1, gave_up)) {
                const int s = t % NS;
                const uint32_t pb = (t % F::pbufs) * F::pbuf;
                fence_after();
                if (issue) {
#pragma unroll
                    for (int k = 0; k < kStep / 16; ++k)
                        mma_ss(tO, dv.at(s * F::stage + k * 16 * 128), dp.at(pb + k * 16 * F::prow), io, done > 0 || k > 0);
                    if (F::rests)
#pragma unroll
                        for (int k = 0; k < kStep / 16; ++k)
                            mma_ss(tO, dv.at(s * F::stage + k * 16 * 128), dp.at(pb + F::p + k * 16 * F::prow), io, true);
                    mma_commit(&bars.empty[s]);
                }
                __syncwarp();
                if (++done == w.steps) {
                    w.next(a);
                    done = 0;
                }
                ++t;
                idle = 0;
            } else if (++idle > kIdle) {
                *gave_up = 1;
            }
        }
        for (int i = max(0, t - NS); i < t; ++i) bar_drain(&bars.empty[i % NS], (i / NS) & 1);
        __syncwarp();
    } else {
        // Group `gr` has rows r0 .. r0 + C - 1 of map m, columns gr * C .. of the
        // scores and sums; a thread has key kr of each step.
        const int gr = warp >> 2, m = gr * C / RT, r0 = gr * C % RT, kr = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float mul = d.scale_log2;
        int t = 0, slot_tile[2] = {-1, -1}, slot_last = 0;
        for (; w.left > 0; w.next(a)) {
            const Tile tile = w.t;
            const int b = tile.b, old = tile.len - tile.count;
            if (kr < C) {
                const int dl = static_cast<int>(d.div_G.div(r0 + kr)), l = min(tile.l0 + dl, d.Lq - 1);
                const int h = min(w.n * d.G + r0 + kr - dl * d.G, d.H - 1);
                row_l[gr][kr] = l;
                row_h[gr][kr] = h;
                row_pos[gr][kr] = d.pos_q ? d.pos_q[static_cast<int64_t>(b) * d.Lq + l] : old + l;
                noff[gr][kr] = FLT_MAX;
                for (int i = 0; i < 2; ++i) far_bias[gr][i][kr] = d.nb ? table[bmap[i * 2 * d.reach] + h] : 0.f;
            }
            // A step ahead: whether the thread's key is to be used, and where it is.
            bool next_use;
            int next_pos;
            const auto fetch = [&](int step) {
                const int j = step * kStep + kr;
                next_use = j < tile.end;
                next_pos = j;
                if (next_use) {
                    const int64_t of = static_cast<int64_t>(b) * d.Lk + j;
                    int place;
                    if (d.pos_k) next_pos = d.pos_k[of];
                    if (d.mask && !d.mask[of]) next_use = false;
                    if (paged_page(d, b, j, place) < 0) next_use = false;
                }
            };
            fetch(w.first);
            sync_group(gr);
            int qmin = INT32_MAX, qmax = INT32_MIN;
            if (lane < C && r0 + lane < used && tile.l0 + static_cast<int>(d.div_G.div(r0 + lane)) < tile.count) qmin = qmax = row_pos[gr][lane];
            qmin = __reduce_min_sync(0xffffffffu, qmin);
            qmax = __reduce_max_sync(0xffffffffu, qmax);
            float sum[C];
#pragma unroll
            for (int c = 0; c < C; ++c) sum[c] = 0.f;
            for (int i = 0; i < w.steps; ++i, ++t) {
                const int s = t % NS, j = (w.first + i) * kStep + kr;
                const bool use = next_use;
                const int pos = next_pos;
                if (i + 1 < w.steps) fetch(w.first + i + 1);
                const bool all = __all_sync(0xffffffffu, use);
                const int64_t kmin = __reduce_min_sync(0xffffffffu, use ? pos : INT32_MAX), kmax = __reduce_max_sync(0xffffffffu, use ? pos : INT32_MIN);
                // Whether every row sees all of the warp's keys, with one bias for each row.
                const bool before = d.nb == 0 || kmax - qmin <= -d.reach, after = !before && kmin - qmax >= d.reach;
                const bool fast = (before || after) && !(d.causal && kmax > qmin) && !(d.pg.tree && (j - lane + 31) >= old);
                bar_wait_warp(&bars.s_full[t & 1], (t >> 1) & 1, gave_up);
                fence_after();
                float x[C];
                // First the scores in base 2 less the rows' references; if some
                // weight would be too large, then the scores alone, for new
                // references, and then once more.
#pragma unroll 1
                for (int pass = 0;; ++pass) {
                    const bool less = pass != 1;
                    tmem_load(tS(0, t) + gr * C + lanes, x);
                    if (fast) {
#pragma unroll
                        for (int c = 0; c < C; c += 4) {
                            float4 o = less ? *reinterpret_cast<const float4 *>(&noff[gr][c]) : make_float4(0.f, 0.f, 0.f, 0.f);
                            if (d.nb) {
                                x[c] = fmaf(x[c], mul, far_bias[gr][after][c]) + o.x;
                                x[c + 1] = fmaf(x[c + 1], mul, far_bias[gr][after][c + 1]) + o.y;
                                x[c + 2] = fmaf(x[c + 2], mul, far_bias[gr][after][c + 2]) + o.z;
                                x[c + 3] = fmaf(x[c + 3], mul, far_bias[gr][after][c + 3]) + o.w;
                            } else {
                                x[c] = fmaf(x[c], mul, o.x);
                                x[c + 1] = fmaf(x[c + 1], mul, o.y);
                                x[c + 2] = fmaf(x[c + 2], mul, o.z);
                                x[c + 3] = fmaf(x[c + 3], mul, o.w);
                            }
                        }
                        if (!all)
#pragma unroll
                            for (int c = 0; c < C; ++c) x[c] = use ? x[c] : -INFINITY;
                    } else {
                        bool leaf = true;
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            const int rel = pos - row_pos[gr][c];
                            if (d.pg.tree && use && j >= old && (c == 0 || row_l[gr][c] != row_l[gr][c - 1]))
                                leaf = d.pg.tree[(static_cast<int64_t>(b) * d.Lq + row_l[gr][c]) * d.Lq + j - old] != 0;
                            const float bias = d.nb ? table[bmap[min(max(rel, -d.reach), d.reach) + d.reach] + row_h[gr][c]] : 0.f;
                            const float y = fmaf(x[c], mul, bias) + (less ? noff[gr][c] : 0.f);
                            x[c] = use && leaf && !(d.causal && rel > 0) ? y : -INFINITY;
                        }
                    }
                    if (pass == 2) break;
                    if (pass == 0) {
                        bool over = false;
#pragma unroll
                        for (int c = 0; c < C; ++c) over |= x[c] > kLift<T> + kSlack;
                        if (!vote(gr, over)) break;
                        continue;
                    }
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const float best = warp_max(x[c]);
                        if (lane == c) wide[gr][warp & 3][c] = best;
                    }
                    sync_group(gr);
                    if (kr < C) {
                        const float best = fmaxf(fmaxf(wide[gr][0][kr], wide[gr][1][kr]), fmaxf(wide[gr][2][kr], wide[gr][3][kr]));
                        const float ref = -noff[gr][kr];
                        const bool raise = best + noff[gr][kr] > kLift<T> + kSlack;
                        const float next = raise ? best - kLift<T> : ref;
                        noff[gr][kr] = -next;
                        shrink[gr][kr] = raise ? ex2(ref - next) : 1.f;
                    }
                    sync_group(gr);
                    if (i > 0) {
                        bar_wait_warp(&bars.empty[(t - 1) % NS], ((t - 1) / NS) & 1, gave_up);
                        fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < C; c0 += 16) {
                            float o[16];
                            tmem_load(tO + gr * C + c0 + lanes, o);
#pragma unroll
                            for (int c = 0; c < 16; ++c) o[c] *= shrink[gr][c0 + c];
                            tmem_store(tO + gr * C + c0 + lanes, o);
                        }
                        tmem_store_wait();
                    }
#pragma unroll
                    for (int c = 0; c < C; ++c) sum[c] *= shrink[gr][c];
                }
                // The weights' buffer is free when the products before have read
                // it: those two steps ago, for which the scores' barrier stands
                // too, or with one buffer those of the last step.
                if (F::pbufs == 1 && t > 0) {
                    bar_wait_warp(&bars.empty[(t - 1) % NS], ((t - 1) / NS) & 1, gave_up);
                }
                unsigned char *pt = base + F::at_p + (t % F::pbufs) * F::pbuf + (RT == 64 ? m * (F::p / 2) : 0) + kr * F::prow;
                const int swz = RT == 16 ? (kr >> 1) & 3 : kr & 7, piece0 = (RT == 64 ? r0 : gr * C) / 8;
#pragma unroll
                for (int c = 0; c < C; c += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float p0 = ex2(x[c + 2 * k]), p1 = ex2(x[c + 2 * k + 1]);
                        sum[c + 2 * k] += p0;
                        sum[c + 2 * k + 1] += p1;
                        hi[k] = pack2<T>(p0, p1);
                        if (F::rests) {
                            const float2 r = unpack2<T>(hi[k]);
                            lo[k] = pack2<T>(p0 - r.x, p1 - r.y);
                        }
                    }
                    const int at = ((piece0 + c / 8) ^ swz) << 4;
                    *reinterpret_cast<uint4 *>(pt + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if (F::rests) *reinterpret_cast<uint4 *>(pt + F::p + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                if (!all && gr < VP / 64) {
                    // 0 * NaN is NaN: unused keys' rows of V become zeros.
                    bar_wait_warp(&bars.full[s], (t / NS) & 1, gave_up);
                    unsigned char *v = base + F::at_stage + s * F::stage + gr * F::vblock + kr * 128;
                    if (!use)
#pragma unroll
                        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(v + (((c + lane) & 7) << 4)) = make_uint4(0, 0, 0, 0);
                }
                fence_async();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bars.p_full[t & 1]);
            }
            // The segment's end: weights' sums over the threads, then the sums themselves.
            fold<C>(sum, lane, 16);
            if (C == 32) wide[gr][warp & 3][lane] = sum[0];
            else if ((lane & 1) == 0) wide[gr][warp & 3][lane >> 1] = sum[0];
            bar_wait_warp(&bars.empty[(t - 1) % NS], ((t - 1) / NS) & 1, gave_up);
            fence_after();
            sync_groups<F::groups * 128>();
            const float nan = *gave_up ? NAN : 0.f;
            const auto whole_sum = [&](int g, int c) { return wide[g][0][c] + wide[g][1][c] + (wide[g][2][c] + wide[g][3][c]) + nan; };
            const int dv = (warp & 3) * 32 + lane;
            if (w.first == 0 && w.steps == tile.steps) {
                // Each group takes its share of the rows, of both maps.
                constexpr int share_rows = RT / F::groups;
#pragma unroll 1
                for (int q0 = gr * share_rows; q0 < (gr + 1) * share_rows; q0 += 8) {
                    float x[8], y[8];
                    __syncwarp();
                    tmem_load(tO + q0 + lanes, x);
                    tmem_load(tO + RT + q0 + lanes, y);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int r = q0 + c, l = tile.l0 + static_cast<int>(d.div_G.div(r));
                        if (r >= used || l >= d.Lq || dv >= d.Dv) continue;
                        const int h = row_h[r / C][r % C];
                        const float s0 = whole_sum(r / C, r % C), s1 = whole_sum(F::groups / 2 + r / C, r % C);
                        const float o = (s0 == 0.f ? 0.f : x[c] / s0) - d.lam[h] * (s1 == 0.f ? 0.f : y[c] / s1);
                        static_cast<T *>(d.out)[((static_cast<int64_t>(b) * d.Lq + l) * d.H + h) * d.Dv + dv] =
                            dattn_round<T>(l < tile.count ? o : 0.f);
                    }
                }
            } else {
                const int k = w.first == 0;
                const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + k;
                slot_tile[k] = w.e * d.Hkv + w.n;
                if (!k) slot_last = w.first + w.steps == tile.steps;
#pragma unroll 1
                for (int c0 = 0; c0 < C; c0 += 8) {
                    float x[8];
                    __syncwarp();
                    tmem_load(tO + gr * C + c0 + lanes, x);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (r0 + c0 + c < used && dv < d.Dv) d.part_o[((slot * RT + r0 + c0 + c) * 2 + m) * d.Dv + dv] = x[c];
                }
                if (kr < C && r0 + kr < used) {
                    float *ml = d.part_ml + ((slot * RT + r0 + kr) * 2 + m) * 2;
                    ml[0] = -noff[gr][kr];
                    ml[1] = whole_sum(gr, kr);
                }
            }
            __syncwarp();
            sync_groups<F::groups * 128>();  // the next segment's arrays are the same
        }
        if (threadIdx.x < 2) {
            a.slots[blockIdx.x * 4 + threadIdx.x * 2] = threadIdx.x ? slot_tile[1] : slot_tile[0];
            a.slots[blockIdx.x * 4 + threadIdx.x * 2 + 1] = slot_last;
        }
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    if (warp == kIssue) {
        fence_after();
        tmem_free(tmem, columns);
    }
    if (threadIdx.x == 0 && *gave_up) atomicOr(&g_paged_gave_up, 1u);
}

// Joins a tile's pieces: the one that begins it is in the second slot of CTA
// blockIdx.x, the others in the first slots of the CTAs after it. A block per
// row, its warps share the pieces.
template <typename T> __global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedTcArgs a, int ctas, int RT)
{
    pdl_wait();
    const DattnArgs &d = a.d;
    const int c = blockIdx.x, r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = a.slots[c * 4 + 2];
    if (tile < 0 || r >= a.LP * d.G) return;
    const int e = tile / d.Hkv, n = tile - e * d.Hkv, b = e / a.row_tiles;
    const int dl = static_cast<int>(d.div_G.div(r)), l = (e - b * a.row_tiles) * a.LP + dl, h = n * d.G + r - dl * d.G;
    if (l >= d.Lq) return;
    int pieces = ctas - c;
    for (int i = 1; i < ctas - c; i += 32) {
        const bool last = i + lane < ctas - c && a.slots[(c + i + lane) * 4 + 1];
        const uint32_t any = __ballot_sync(0xffffffffu, last);
        if (any) {
            pieces = i + __ffs(any);
            break;
        }
    }
    const auto slot = [&](int i) { return i == 0 ? static_cast<int64_t>(c) * 2 + 1 : static_cast<int64_t>(c + i) * 2; };
    const auto ml = [&](int i, int m) { return *reinterpret_cast<const float2 *>(d.part_ml + ((slot(i) * RT + r) * 2 + m) * 2); };
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    for (int i = lane; i < pieces; i += 32)
        for (int m = 0; m < 2; ++m) top[m] = fmaxf(top[m], ml(i, m).x);
    for (int m = 0; m < 2; ++m) {
        for (int o = 16; o; o >>= 1) top[m] = fmaxf(top[m], __shfl_xor_sync(0xffffffffu, top[m], o));
        for (int i = lane; i < pieces; i += 32) {
            const float2 x = ml(i, m);
            sum[m] = fmaf(x.y, ex2(x.x - top[m]), sum[m]);
        }
        for (int o = 16; o; o >>= 1) sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], o);
    }
    __shared__ float part[8][2][128];
    const int v = lane * 4;
    float4 o[2] = {};
    if (v < d.Dv)
        for (int i = warp; i < pieces; i += 8)
            for (int m = 0; m < 2; ++m) {
                const float f = ex2(ml(i, m).x - top[m]);
                const float4 x = *reinterpret_cast<const float4 *>(d.part_o + ((slot(i) * RT + r) * 2 + m) * d.Dv + v);
                o[m].x = fmaf(x.x, f, o[m].x);
                o[m].y = fmaf(x.y, f, o[m].y);
                o[m].z = fmaf(x.z, f, o[m].z);
                o[m].w = fmaf(x.w, f, o[m].w);
            }
    for (int m = 0; m < 2; ++m) *reinterpret_cast<float4 *>(&part[warp][m][v]) = o[m];
    __syncthreads();
    if (static_cast<int>(threadIdx.x) >= d.Dv) return;
    float x[2] = {0.f, 0.f};
    for (int m = 0; m < 2; ++m)
        for (int i = 0; i < 8; ++i) x[m] += part[i][m][threadIdx.x];
    const float out = (sum[0] == 0.f ? 0.f : x[0] / sum[0]) - d.lam[h] * (sum[1] == 0.f ? 0.f : x[1] / sum[1]);
    static_cast<T *>(d.out)[((static_cast<int64_t>(b) * d.Lq + l) * d.H + h) * d.Dv + threadIdx.x] =
        dattn_round<T>(l < paged_count(d, b) ? out : 0.f);
}

template <typename T, int DP, int VP, int RT>
cudaError_t launch_tc(const PagedTcArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st)
{
    using F = PgShared<DP, VP, RT>;
    const size_t smem = F::bytes + 1024 + paged_bias_bytes(a.d.nb, a.d.H, a.d.reach);
    const auto kernel = paged_tc_kernel<T, DP, VP, RT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    kernel<<<a.ctas, F::threads, smem, st>>>(a, mq, mk, mv);
    e = cudaGetLastError();
    if (e == cudaSuccess && a.ctas > 1)  // one CTA has no pieces
        e = launch_pdl(paged_join_kernel<T>, dim3(a.ctas, a.LP * a.d.G), dim3(256), 0, st, a, a.ctas, RT);
    return e;
}

template <typename T, int DP, int VP>
cudaError_t any_rows(const PagedTcArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st)
{
    return a.RT == 16 ? launch_tc<T, DP, VP, 16>(a, mq, mk, mv, st) : a.RT == 32 ? launch_tc<T, DP, VP, 32>(a, mq, mk, mv, st)
                                                                               : launch_tc<T, DP, VP, 64>(a, mq, mk, mv, st);
}

template <typename T>
cudaError_t any_width(const PagedTcArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st)
{
    return a.d.D <= 32 && a.d.Dv <= 64 ? any_rows<T, 32, 64>(a, mq, mk, mv, st) : any_rows<T, 64, 128>(a, mq, mk, mv, st);
}

template <typename T> da_status forward_tensor(const PagedTcArgs &a, int dtype, cudaStream_t st)
{
    const DattnArgs &d = a.d;
    const int wide = d.D <= 32 && d.Dv <= 64 ? 32 : 64;  // as any_width has it
    CUtensorMap mq, mk, mv;
    da_status e = tensor_map(mq, dtype, d.q, d.D, 2, d.H, d.Lq, d.B, d.qs[3], d.qs[2], d.qs[1], d.qs[0], wide, d.G, a.LP);
    if (e == DA_OK)
        e = tensor_map(mk, dtype, d.k, d.D, 2, d.Hkv, d.pg.page_size, d.pg.num_pages, d.ks[3], d.ks[2], d.ks[1], d.ks[0], wide, 1, a.box);
    if (e == DA_OK)
        e = tensor_map(mv, dtype, d.v, d.Dv, 1, d.Hkv, d.pg.page_size, d.pg.num_pages, 0, d.vs[2], d.vs[1], d.vs[0], 64, 1, a.box);
    if (e != DA_OK) return e;
    const cudaError_t c = any_width<T>(a, mq, mk, mv, st);
    return c == cudaSuccess ? DA_OK : cuda_fail(c, "paged attention launch");
}

uint32_t *gave_up_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_paged_gave_up) == cudaSuccess ? static_cast<uint32_t *>(p) : nullptr;
}

}  // namespace
}  // namespace da
