// Differential attention over a paged cache on the tensor cores
// (include/paged.h), for bf16 and fp16: O = P_0 V - lam P_1 V, P_m the softmax of
// scale K_m q_m^T and the bias over the keys that a row sees, in one pass with a
// running reference for its maximum.
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
// Warps: 0-3 make the weights of map 0 and 4-7 of map 1, 8 loads keys by TMA and 10
// values (a box lies in one page: gcd(page size, 128) places), 9 issues the scores'
// products and 11 the sums', each as soon as what it needs is there. Weights go
// through shared memory, rounded to the inputs' type. Tiles of 16 and 32 rows,
// which take up to 64 rows and which memory bounds, carry what that rounding took
// as a second operand, so that their outputs are off by one rounding (2-norm
// 0.0017 in bf16, 0.00021 in fp16). With tiles of 64 rows outputs have the error of
// two independent roundings, 1.55 times that (0.0026 and 0.00032): a second operand
// there took 222 us where one took 126, in a replayed graph at 1,021 tokens over
// 8,001 keys.
//
// Measured, a call among others, with the kernel that joins pieces:
// - a token each over eight caches of up to 32,768 keys (16 heads, 4 key heads,
//   D = 64, bf16): 80 us, 5.3 TB/s of the 6.8 that a copy reaches; memory bounds
//   it (DRAM 67 % busy from a cold L2), then the uneven ends and the join (6 us).
//   Keys and values have rings of their own because values are needed later;
// - 31 drafted tokens over four caches of 8,191 keys (fp16): 31 us, six steps
//   for a CTA, so set-up, beginnings, ends and the join (7 us) are most of it;
// - 1,021 tokens over 8,001 keys twice (8 heads, 2 key heads): 120 us. A step of
//   128 keys and 64 rows of both maps takes some 2,000 clocks, 1,000 of them of
//   products; its 16,384 exponentials would take 512. What is left is the
//   chain of a step: wait, read scores, weights, vote, fence, arrive. 16 warps to
//   make weights take 151 us (their barriers cost more than they hide), scores
//   16, 32 or 64 at once and loops rolled or not 124 to 127.
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

// Shared memory: q, then rings of values and of keys, then weights. With VP = 64
// the product's second 64 rows, which nothing reads, are whatever follows a
// stage of values.
template <int DP, int VP, int RT> struct PgShared {
    static constexpr int row = DP * 2;                   // bytes of a row of q or k
    static constexpr int q = RT * row;                   // of one map
    static constexpr int kmap = kStep * row;             // of one map's keys of a step
    static constexpr int k = 2 * kmap;
    static constexpr int vblock = kStep * 128;           // of 64 columns of V
    static constexpr int v = VP / 64 * vblock;
    static constexpr bool rests = RT <= 32;              // weights carry what rounding took
    static constexpr int prow = RT == 16 ? 64 : 128;     // bytes of a key's row of weights
    static constexpr int p = kStep * 2 * RT * 2;         // of both maps' weights
    static constexpr int pbuf = p * (rests ? 2 : 1);
    // Steps that each ring holds, and the weights' buffers: what 227 KB allow.
    // Values stay longer than keys, until a step's weights are made.
    static constexpr int ks = DP == 32 ? 4 : RT == 16 ? 3 : 2, vs = DP == 32 ? 4 : RT <= 32 ? 3 : 2;
    static constexpr int pbufs = RT == 64 || DP == 32 ? 2 : 1;
    static constexpr int at_v = 2 * q, at_k = at_v + vs * v, at_p = at_k + ks * k, bytes = at_p + pbufs * pbuf;
    static constexpr int arrays = RT * 128 + 4096;     // the kernel's static ones, at most
    static_assert(bytes + 1024 + kPgBias + arrays <= 227 * 1024, "shared memory");
};

constexpr int kInfos = 6;  // of the steps' infos: two more than keys are ahead of the weights made from them

// What passes a phase ahead has a barrier for even and one for odd steps; the
// others' next phase cannot end before everyone has seen the last one.
struct PgBars {
    uint64_t q_full, q_empty;
    uint64_t k_full[4], k_empty[4];  // empty: the step's scores are done
    uint64_t v_full[4], v_empty[4];  // empty: its sums are done, and its weights' buffer is free
    uint64_t s_full[2], p_full[2];   // scores, weights
    uint32_t tmem, gave_up;
};

__device__ uint32_t g_paged_gave_up;

// A tile of a sequence's rows (all key heads have the same).
struct Tile {
    int b, l0, len, count, end, steps;  // sequence, first query, keys, queries, keys that some query sees, steps of them
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
    t.steps = (t.end + kStep - 1) / kStep;
    return t;
}

// What a tile costs, in steps: to begin and end one takes as long as kOpen. (With
// 0 instead the trees and prompts above take 40 and 132 us instead of 35 and
// 125 in a replayed graph; with 2 or 8 38 and 35, 126 and 125.)
constexpr int kOpen = 4;
__device__ __forceinline__ int units(const Tile &t) { return t.steps ? t.steps + kOpen : 0; }

// A CTA's walk over its share of units, segment by segment: `steps` of tile
// (e, n) from `first` on. Units that only open a tile bring no segment.
struct Walk {
    int64_t left;
    int e, n, at, first, steps;
    Tile t;

    __device__ __forceinline__ void settle(const PagedTcArgs &a)
    {
        while (left > 0) {
            if (t.steps > 0) {
                const int64_t to = min(static_cast<int64_t>(units(t)), at + left);
                first = max(at - kOpen, 0);
                steps = static_cast<int>(max(to - kOpen, int64_t{0})) - first;
                if (steps > 0) return;
            }
            pass(a);
        }
    }
    __device__ __forceinline__ void pass(const PagedTcArgs &a)
    {
        left -= units(t) - at;
        at = 0;
        if (left <= 0) return;
        if (t.steps == 0 || ++n == a.d.Hkv) {
            n = 0;
            t = tile_of(a, ++e);
        }
    }
    __device__ __forceinline__ void start(const PagedTcArgs &a, int64_t share, int e_, int n_, int at_)
    {
        left = share;
        e = e_;
        n = n_;
        at = at_;
        if (left <= 0) return;
        t = tile_of(a, e);
        settle(a);
    }
    __device__ __forceinline__ void next(const PagedTcArgs &a)
    {
        pass(a);
        settle(a);
    }
};

constexpr int kFar = 1 << 30;  // beyond every position

// What is known of a step's keys, by groups of 32: which are to be used, and
// the least and largest of their positions.
struct StepInfo {
    uint32_t use[4];
    int lo[4], hi[4];
};

// Whether any of the 128 threads of map m has `flag`.
__device__ __forceinline__ bool vote(int m, bool flag)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                 "bar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(static_cast<uint32_t>(flag)), "r"(1 + m)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_map(int m) { asm volatile("bar.sync %0, 128;" ::"r"(1 + m) : "memory"); }
__device__ __forceinline__ void sync_maps() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

// Maximum over the warp; a NaN counts for nothing.
__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

constexpr int kPgThreads = 12 * 32;

// Weights are summed by a product with ones, as the products take them, so that
// numerator and denominator have the same roundings. Sums by the threads, which
// read back their weights, cost 300 instructions and 64 registers of a thread at
// 64 rows: 1,021 new tokens over 8,001 keys took 149 us with them, 126 without.
// The operand of [128, 16] ones: its blocks of 8 rows by 16 bytes begin 16 bytes
// after one another, so that 16 by 2 of them take 384 bytes.
constexpr int kOnes = 192;
__device__ __forceinline__ uint64_t ones_operand(const void *ones)
{
    return static_cast<uint64_t>((1u << 14) | 1u) << 32 | (smem_addr(ones) >> 4 | (1u << 16));
}

template <typename T, int DP, int VP, int RT>
__global__ void __launch_bounds__(kPgThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedTcArgs a, const __grid_constant__ CUtensorMap mq,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv)
{
    using F = PgShared<DP, VP, RT>;
    constexpr int NK = F::ks, NV = F::vs;
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t columns = RT == 16 ? 128 : RT == 32 ? 256 : 512;
    extern __shared__ unsigned char raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    __shared__ PgBars bars;
    __shared__ StepInfo infos[kInfos];
    __shared__ int key_pos[kInfos][kStep];                 // where positions are given
    // Each map's rows.
    __shared__ __align__(16) float noff[2][RT];            // minus the row's reference
    __shared__ __align__(16) float off[2][2][RT];          // the same, with far_bias
    __shared__ __align__(16) float shrink[2][RT];
    __shared__ __align__(16) float wide[2][4][RT];         // a warp's maxima; weights' sums in [0]
    __shared__ __align__(16) float far_bias[2][2][RT];     // of keys `reach` or more before and after the query
    __shared__ __align__(16) int row_pos[2][RT], row_l[2][RT], row_h[2][RT];
    __shared__ uint64_t row_tree[2][RT];                   // which of at most 64 new tokens the row sees
    __shared__ int64_t row_out[RT];                        // where the row's output is, or -1
    __shared__ int64_t warp_total[kPgThreads / 32];
    __shared__ int start[3];
    __shared__ __align__(16) T ones[kOnes];
    float *table = reinterpret_cast<float *>(base + F::bytes);  // [nb][H], times log2(e)
    uint16_t *bmap = reinterpret_cast<uint16_t *>(table + a.d.nb * a.d.H);
    const DattnArgs &d = a.d;
    const int warp = warp_number(), lane = threadIdx.x & 31;
    pdl_trigger();  // the kernel that joins the pieces waits for this one's end, but not to be launched

    if (threadIdx.x == 0) {
        bar_init(&bars.q_full, 1);
        bar_init(&bars.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(&bars.s_full[i], 1);
            bar_init(&bars.p_full[i], 8);
        }
        for (int s = 0; s < 4; ++s) {
            bar_init(&bars.k_full[s], 1);
            bar_init(&bars.k_empty[s], 1);
            bar_init(&bars.v_full[s], 1);
            bar_init(&bars.v_empty[s], 1);
        }
        bars.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
    }
    if (warp == 9) tmem_alloc(&bars.tmem, columns);
    for (int i = threadIdx.x; i < d.nb * d.H; i += kPgThreads) table[i] = d.table[i] * kLog2e;
    for (int i = threadIdx.x; i < 2 * d.reach + 1 && d.nb; i += kPgThreads)
        bmap[i] = static_cast<uint16_t>(min(max(d.bmap[i], 0), d.nb - 1) * d.H);
    if (threadIdx.x < kOnes) ones[threadIdx.x] = dattn_round<T>(1.f);
    // Rows of q that a tile's queries leave free.
    const int used = a.LP * d.G;
    for (int i = threadIdx.x; i < 2 * (RT - used) * (F::row / 16); i += kPgThreads) {
        const int m = i >= (RT - used) * (F::row / 16), rest = i - m * (RT - used) * (F::row / 16);
        *reinterpret_cast<uint4 *>(base + m * F::q + used * F::row + rest * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async();

    const int entries = d.B * a.row_tiles;
    // The CTA's share: threads take consecutive tiles' units, a scan adds them up.
    const int per = (entries + kPgThreads - 1) / kPgThreads;
    const int e0 = min(static_cast<int>(threadIdx.x) * per, entries), e1 = min(e0 + per, entries);
    int64_t own = 0;
    for (int e = e0; e < e1; ++e) own += units(tile_of(a, e));
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
    for (int w = 0; w < kPgThreads / 32; ++w) {
        if (w == warp) upto += total;
        total += warp_total[w];
    }
    // CTAs without a share are the last ones, so that a tile's pieces lie in CTAs in a row.
    const int64_t active = max(min(total, static_cast<int64_t>(gridDim.x)), int64_t{1}), cta = min(static_cast<int64_t>(blockIdx.x), active);
    const int64_t each = total < INT32_MAX ? static_cast<uint32_t>(total) / static_cast<uint32_t>(active) : total / active;
    const int64_t more = total - each * active, from = each * cta + min(cta, more), share = cta < active ? each + (cta < more) : 0;
    if (share > 0 && from < upto && from >= upto - own) {
        int64_t at = upto - own;
        int e = e0, u = 0;
        for (;; ++e) {
            u = units(tile_of(a, e));
            if (from < at + static_cast<int64_t>(u) * d.Hkv) break;
            at += static_cast<int64_t>(u) * d.Hkv;
        }
        start[0] = e;
        start[1] = static_cast<int>((from - at) / u);
        start[2] = static_cast<int>((from - at) % u);
    }
    __syncthreads();
    const uint32_t tmem = uniform(bars.tmem);
    volatile uint32_t *gave_up = &bars.gave_up;
    const auto tS = [&](int m, int t) { return tmem + ((t & 1) * 2 + m) * RT; };
    const uint32_t tO = tmem + 4 * RT, tL = tO + 2 * RT, sb = smem_addr(base);  // outputs' sums, weights' sums
    Walk w;
    w.start(a, share, start[0], start[1], start[2]);

    if (warp == 8 || warp == 10) {
        // Copies of keys (and queries), and of values: a lane brings one box of a step.
        const bool keys = warp == 8;
        const int boxes = kStep / a.box, blocks = (d.Dv + 63) / 64;
        int t = 0, seg = 0;
        for (; w.left > 0; w.next(a), ++seg) {
            if (keys) {
                bar_wait_warp(&bars.q_empty, (seg & 1) ^ 1, gave_up);
                if (lane == 0) {
                    bar_expect(&bars.q_full, 2 * F::row * used);
                    for (int m = 0; m < 2; ++m) tma_load(&mq, &bars.q_full, base + m * F::q, 0, m, w.n * d.G, w.t.l0, w.t.b);
                }
            }
            for (int i = 0; i < w.steps; ++i, ++t) {
                const int j0 = (w.first + i) * kStep, j = j0 + lane * a.box;
                int place = 0, page = -1;
                if (lane < boxes && j < w.t.end) page = paged_page(d, w.t.b, j, place);
                const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
                // The copies are issued before their bytes are expected, with
                // which the phase's only arrival comes.
                if (!keys) {
                    const int s = t % NV;
                    bar_wait_warp(&bars.v_empty[s], ((t / NV) & 1) ^ 1, gave_up);
                    if (page >= 0)
                        for (int c = 0; c < blocks; ++c)
                            tma_load(&mv, &bars.v_full[s], base + F::at_v + s * F::v + c * F::vblock + lane * a.box * 128, c * 64, 0, w.n, place, page);
                    __syncwarp();
                    if (lane == 0) bar_expect(&bars.v_full[s], __popc(there) * a.box * blocks * 128);
                    __syncwarp();
                    continue;
                }
                const int s = t % NK;
                uint32_t used_keys[4];
                int pos[4], lo[4], hi[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int r = g * 32 + lane;
                    bool use = j0 + r < w.t.end && (there >> (r / a.box) & 1);
                    const int64_t of = static_cast<int64_t>(w.t.b) * d.Lk + j0 + r;
                    if (use && d.mask) use = d.mask[of] != 0;
                    pos[g] = use && d.pos_k ? d.pos_k[of] : j0 + r;
                    used_keys[g] = __ballot_sync(0xffffffffu, use);
                    lo[g] = __reduce_min_sync(0xffffffffu, use ? pos[g] : kFar);
                    hi[g] = __reduce_max_sync(0xffffffffu, use ? pos[g] : -kFar);
                }
                bar_wait_warp(&bars.k_empty[s], ((t / NK) & 1) ^ 1, gave_up);
                if (page >= 0)
                    for (int m = 0; m < 2; ++m)
                        tma_load(&mk, &bars.k_full[s], base + F::at_k + s * F::k + m * F::kmap + lane * a.box * F::row, 0, m, w.n, place, page);
                // Their last reader, the weights of kInfos steps ago, came before the scores that freed the keys' place.
                StepInfo &info = infos[t % kInfos];
                if (lane < 4) {
                    info.use[lane] = lane == 0 ? used_keys[0] : lane == 1 ? used_keys[1] : lane == 2 ? used_keys[2] : used_keys[3];
                    info.lo[lane] = lane == 0 ? lo[0] : lane == 1 ? lo[1] : lane == 2 ? lo[2] : lo[3];
                    info.hi[lane] = lane == 0 ? hi[0] : lane == 1 ? hi[1] : lane == 2 ? hi[2] : hi[3];
                }
                if (d.pos_k)
#pragma unroll
                    for (int g = 0; g < 4; ++g) key_pos[t % kInfos][g * 32 + lane] = pos[g];
                __syncwarp();
                if (lane == 0) bar_expect(&bars.k_full[s], __popc(there) * a.box * 2 * F::row);
                __syncwarp();
            }
        }
        if (*gave_up) {  // leave no copy in flight
            if (keys && seg > 0) bar_drain(&bars.q_full, (seg - 1) & 1);
            const int n = keys ? NK : NV;
            for (int i = max(0, t - n); i < t; ++i) bar_drain(keys ? &bars.k_full[i % n] : &bars.v_full[i % n], (i / n) & 1);
        }
    } else if (warp == 9) {
        // Scores. (All lanes walk through the steps, one issues: addresses then
        // stay in uniform registers.)
        const bool issue = elect();
        constexpr uint32_t is = shape(bf16, RT, false);
        const Operand<F::row> dk = along_row<F::row>(sb + F::at_k), dq = along_row<F::row>(sb);
        int t = 0, seg = 0;
        for (; w.left > 0; w.next(a), ++seg) {
            bar_wait_warp(&bars.q_full, seg & 1, gave_up);
            for (int i = 0; i < w.steps; ++i, ++t) {
                const int s = t % NK;
                bar_wait_warp(&bars.k_full[s], (t / NK) & 1, gave_up);
                // Into the columns of two steps ago, which its weights have read.
                if (t > 1) bar_wait_warp(&bars.p_full[t & 1], ((t >> 1) & 1) ^ 1, gave_up);
                fence_after();
                if (issue) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int c = 0; c < DP / 16; ++c)
                            mma_ss(tS(m, t), dk.at(s * F::k + m * F::kmap + c * 32), dq.at(m * F::q + c * 32), is, c > 0);
                    mma_commit(&bars.s_full[t & 1]);
                    mma_commit(&bars.k_empty[s]);
                    if (i == w.steps - 1) mma_commit(&bars.q_empty);
                }
                __syncwarp();
            }
        }
        for (int i = max(0, t - NK); i < t; ++i) bar_drain(&bars.k_empty[i % NK], (i / NK) & 1);
        __syncwarp();
    } else if (warp == 11) {
        // Sums.
        const bool issue = elect();
        constexpr uint32_t il = shape(bf16, 2 * RT, true), io = il | (1u << 15);
        const uint64_t all = ones_operand(ones);
        const Operand<128> dv = over_rows<128>(sb + F::at_v, F::vblock);
        const Operand<F::prow> dp = over_rows<F::prow>(sb + F::at_p, F::p / 2);
        int t = 0;
        for (; w.left > 0; w.next(a)) {
            for (int i = 0; i < w.steps; ++i, ++t) {
                const int s = t % NV;
                const uint32_t pb = (t % F::pbufs) * F::pbuf;
                bar_wait_warp(&bars.v_full[s], (t / NV) & 1, gave_up);
                bar_wait_warp(&bars.p_full[t & 1], (t >> 1) & 1, gave_up);
                fence_after();
                if (issue) {
#pragma unroll
                    for (int c = 0; c < kStep / 16; ++c)
                        mma_ss(tO, dv.at(s * F::v + c * 16 * 128), dp.at(pb + c * 16 * F::prow), io, i > 0 || c > 0);
                    if (F::rests)
#pragma unroll
                        for (int c = 0; c < kStep / 16; ++c)
                            mma_ss(tO, dv.at(s * F::v + c * 16 * 128), dp.at(pb + F::p + c * 16 * F::prow), io, true);
#pragma unroll
                    for (int c = 0; c < kStep / 16; ++c) mma_ss(tL, all, dp.at(pb + c * 16 * F::prow), il, i > 0 || c > 0);
                    if (F::rests)
#pragma unroll
                        for (int c = 0; c < kStep / 16; ++c) mma_ss(tL, all, dp.at(pb + F::p + c * 16 * F::prow), il, true);
                    mma_commit(&bars.v_empty[s]);
                }
                __syncwarp();
            }
        }
        for (int i = max(0, t - NV); i < t; ++i) bar_drain(&bars.v_empty[i % NV], (i / NV) & 1);
        __syncwarp();
    } else {
        // A thread has key kr of each step, and that key's scores of map m with all rows.
        // Scores that it takes at once, and where nothing is masked.
        constexpr int X = 16, XF = RT < 32 ? RT : 32;
        const int m = warp >> 2, kr = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float2 mul = {d.scale_log2, d.scale_log2};
        // The sums with weights of step `of` are done.
        const auto summed = [&](int of) { bar_wait_warp(&bars.v_empty[of % NV], (of / NV) & 1, gave_up); };
        // Rows that see nothing: all heads' outputs of such tiles lie in a row.
        for (int e = blockIdx.x; e < entries; e += gridDim.x) {
            const Tile none = tile_of(a, e);
            if (none.steps) continue;
            T *to = static_cast<T *>(d.out) + (static_cast<int64_t>(none.b) * d.Lq + none.l0) * d.H * d.Dv;
            const int n = min(a.LP, d.Lq - none.l0) * d.H * d.Dv;
            for (int i = threadIdx.x; i < n; i += 256) to[i] = dattn_round<T>(0.f);
        }
        const bool few = d.pg.tree && d.Lq <= 64;  // the tree's rows are bits in shared memory
        int t = 0, slot_tile[2] = {-1, -1}, slot_last = 0;
        for (; w.left > 0; w.next(a)) {
            const Tile tile = w.t;
            const int b = tile.b, old = tile.len - tile.count;
            if (const int r = kr; r < RT) {
                const int dl = static_cast<int>(d.div_G.div(r)), l = min(tile.l0 + dl, d.Lq - 1), h = min(w.n * d.G + r - dl * d.G, d.H - 1);
                row_l[m][r] = l;
                row_h[m][r] = h;
                row_pos[m][r] = d.pos_q ? d.pos_q[static_cast<int64_t>(b) * d.Lq + l] : old + l;
                noff[m][r] = FLT_MAX;
                for (int i = 0; i < 2; ++i) far_bias[m][i][r] = d.nb ? table[bmap[i * 2 * d.reach] + h] : 0.f;
                if (m == 0) row_out[r] = r < used && tile.l0 + dl < d.Lq ? ((static_cast<int64_t>(b) * d.Lq + l) * d.H + h) * d.Dv : -1;
            }
            if (few && (w.first + w.steps) * kStep > old)
                for (int r = warp & 3; r < used; r += 4) {
                    const int l = min(tile.l0 + static_cast<int>(d.div_G.div(r)), d.Lq - 1);
                    const uint8_t *of = d.pg.tree + (static_cast<int64_t>(b) * d.Lq + l) * d.Lq;
                    const uint32_t low = __ballot_sync(0xffffffffu, lane < d.Lq && of[lane]), high = __ballot_sync(0xffffffffu, lane + 32 < d.Lq && of[lane + 32]);
                    if (lane == 0) row_tree[m][r] = low | static_cast<uint64_t>(high) << 32;
                }
            sync_map(m);
            int qmin = kFar, qmax = -kFar;
#pragma unroll
            for (int r = lane; r < RT; r += 32)
                if (r < used && tile.l0 + static_cast<int>(d.div_G.div(r)) < tile.count) {
                    qmin = min(qmin, row_pos[m][r]);
                    qmax = max(qmax, row_pos[m][r]);
                }
            qmin = __reduce_min_sync(0xffffffffu, qmin);
            qmax = __reduce_max_sync(0xffffffffu, qmax);
#pragma unroll 1
            for (int i = 0; i < w.steps; ++i, ++t) {
                const int j = (w.first + i) * kStep + kr;
                bar_wait_warp(&bars.s_full[t & 1], (t >> 1) & 1, gave_up);
                fence_after();
                const StepInfo &info = infos[t % kInfos];
                const uint32_t used_keys = info.use[warp & 3];
                const bool use = used_keys >> lane & 1, all = used_keys == 0xffffffffu;
                const int pos = d.pos_k ? key_pos[t % kInfos][kr] : j, kmin = info.lo[warp & 3], kmax = info.hi[warp & 3];
                // Whether every row sees all of the warp's keys, with one bias for each row.
                const bool before = d.nb == 0 || kmax - qmin <= -d.reach, after = !before && kmin - qmax >= d.reach;
                const bool fast = (before || after) && !(d.causal && kmax > qmin) && !(d.pg.tree && (j - lane + 31) >= old);
                // Scores of rows c0 .. in base 2, less the rows' references (or not).
                const auto finish = [&](float (&x)[X], int c0, bool less) {
                    uint32_t see = use ? 0xffffffffu : 0u;
                    if (d.causal)
#pragma unroll
                        for (int c = 0; c < X; ++c)
                            if (pos > row_pos[m][c0 + c]) see &= ~(1u << c);
                    if (d.pg.tree && use && j >= old) {
                        if (few) {
#pragma unroll
                            for (int c = 0; c < X; ++c)
                                if (!(row_tree[m][c0 + c] >> (j - old) & 1)) see &= ~(1u << c);
                        } else {
#pragma unroll
                            for (int c = 0; c < X; ++c)
                                if (!d.pg.tree[(static_cast<int64_t>(b) * d.Lq + row_l[m][c0 + c]) * d.Lq + j - old]) see &= ~(1u << c);
                        }
                    }
                    float bias[X];
                    if (fast || d.nb == 0) {
#pragma unroll
                        for (int c = 0; c < X; ++c) bias[c] = far_bias[m][after][c0 + c];
                    } else {
#pragma unroll
                        for (int c = 0; c < X; ++c)
                            bias[c] = table[bmap[min(max(pos - row_pos[m][c0 + c], -d.reach), d.reach) + d.reach] + row_h[m][c0 + c]];
                    }
#pragma unroll
                    for (int c = 0; c < X; ++c) {
                        const float y = fmaf(x[c], mul.x, bias[c]) + (less ? noff[m][c0 + c] : 0.f);
                        x[c] = see >> c & 1 ? y : -INFINITY;
                    }
                };
                // The step's weights; once more where one would be too large for
                // its row's reference. A segment begins with references. Weights go
                // to shared memory at once; sums take them from there when they stand.
                if (t >= F::pbufs) summed(t - F::pbufs);  // the weights' buffer is free
                const int swz = RT == 16 ? (kr >> 1) & 3 : kr & 7, piece0 = RT == 64 ? 0 : m * RT / 8;
                unsigned char *const pt = base + F::at_p + (t % F::pbufs) * F::pbuf + (RT == 64 ? m * (F::p / 2) : 0) + kr * F::prow;
                const auto piece = [&](int c) { return reinterpret_cast<uint4 *>(pt + (((piece0 + c / 8) ^ swz) << 4)); };
                const auto weigh = [&](const auto &x, int c0) {
#pragma unroll
                    for (int c = 0; c < static_cast<int>(sizeof(x) / sizeof(float)); c += 8) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 w2 = {ex2(x[c + 2 * k]), ex2(x[c + 2 * k + 1])};
                            hi[k] = pack2<T>(w2.x, w2.y);
                            if constexpr (F::rests) {
                                const float2 r = unpack2<T>(hi[k]);
                                lo[k] = pack2<T>(w2.x - r.x, w2.y - r.y);
                            }
                        }
                        *piece(c0 + c) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        if constexpr (F::rests) piece(c0 + c)[F::p / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                };
                const uint32_t scores = tS(m, t) + lanes;
#pragma unroll 1
                for (bool again = false;; again = true) {
                    float top[2] = {-INFINITY, -INFINITY};
                    if (i == 0 && !again) {
                        top[0] = INFINITY;
                    } else if (fast && all) {
                        // Most steps: no branches, for the sake of the order of instructions.
                        const float *o = &off[m][after][0];
#pragma unroll 1
                        for (int c0 = 0; c0 < RT; c0 += XF) {
                            float x[XF];
                            tmem_load(scores + c0, x);
#pragma unroll
                            for (int c = 0; c < XF; c += 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(o + c0 + c);
                                const float2 u = fma2({x[c], x[c + 1]}, mul, {f.x, f.y}), v = fma2({x[c + 2], x[c + 3]}, mul, {f.z, f.w});
                                x[c] = u.x;
                                x[c + 1] = u.y;
                                x[c + 2] = v.x;
                                x[c + 3] = v.y;
                                top[0] = max3(top[0], u.x, u.y);
                                top[1] = max3(top[1], v.x, v.y);
                            }
                            weigh(x, c0);
                        }
                    } else {
#pragma unroll 1
                        for (int c0 = 0; c0 < RT; c0 += X) {
                            float x[X];
                            tmem_load(scores + c0, x);
                            finish(x, c0, true);
#pragma unroll
                            for (int c = 0; c < X; c += 2) top[0] = max3(top[0], x[c], x[c + 1]);
                            weigh(x, c0);
                        }
                    }
                    if (again || (i > 0 && !vote(m, fmaxf(top[0], top[1]) > kLift<T> + kSlack))) break;
#pragma unroll 1
                    for (int c0 = 0; c0 < RT; c0 += X) {
                        float x[X];
                        tmem_load(scores + c0, x);
                        finish(x, c0, false);
                        float best = -INFINITY;  // of row c0 + lane
#pragma unroll
                        for (int c = 0; c < X; ++c) {
                            const float of = warp_max(x[c]);
                            best = lane == c ? of : best;
                        }
                        if (lane < X) wide[m][warp & 3][c0 + lane] = best;
                    }
                    sync_map(m);
                    if (const int r = kr; r < RT) {
                        const float best = fmaxf(fmaxf(wide[m][0][r], wide[m][1][r]), fmaxf(wide[m][2][r], wide[m][3][r]));
                        const float ref = -noff[m][r];
                        const bool raise = best + noff[m][r] > kLift<T> + kSlack;
                        const float next = raise ? best - kLift<T> : ref;
                        noff[m][r] = -next;
                        for (int k = 0; k < 2; ++k) off[m][k][r] = far_bias[m][k][r] - next;
                        shrink[m][r] = raise ? ex2(ref - next) : 1.f;
                    }
                    sync_map(m);
                    if (i > 0) {
                        summed(t - 1);
                        fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < 2 * RT; c0 += 16) {
                            const uint32_t at = (c0 < RT ? tO + c0 : tL + c0 - RT) + m * RT + lanes;
                            float o[16];
                            tmem_load(at, o);
#pragma unroll
                            for (int c = 0; c < 16; ++c) o[c] *= shrink[m][(c0 + c) % RT];
                            tmem_store(at, o);
                        }
                        tmem_store_wait();
                    }
                }
                if (!all && m < VP / 64) {
                    // 0 * NaN is NaN: unused keys' rows of V become zeros.
                    bar_wait_warp(&bars.v_full[t % NV], (t / NV) & 1, gave_up);
                    unsigned char *v = base + F::at_v + (t % NV) * F::v + m * F::vblock + kr * 128;
                    if (!use)
#pragma unroll
                        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(v + (((c + lane) & 7) << 4)) = make_uint4(0, 0, 0, 0);
                }
                fence_async();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bars.p_full[t & 1]);
            }
            summed(t - 1);
            fence_after();
            if ((warp & 3) == 0)
#pragma unroll 1
                for (int c0 = 0; c0 < RT; c0 += 16) {
                    float l[16];
                    __syncwarp();
                    tmem_load(tL + m * RT + c0, l);
                    if (lane == 0)
#pragma unroll
                        for (int c = 0; c < 16; ++c) wide[m][0][c0 + c] = l[c];
                }
            sync_maps();
            const bool whole = w.first == 0 && w.steps == tile.steps;
            const int dv = (warp & 3) * 32 + lane, k = w.first == 0;
            const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + k;
            if (const int r = kr; r < RT) {
                const float total = wide[m][0][r] + (*gave_up ? NAN : 0.f);
                if (whole) {
                    shrink[m][r] = total == 0.f || row_l[m][r] >= tile.count ? 0.f : (m ? d.lam[row_h[m][r]] : 1.f) / total;
                } else if (r < used) {
                    *reinterpret_cast<float2 *>(d.part_ml + ((slot * RT + r) * 2 + m) * 2) = make_float2(-noff[m][r], total);
                }
            }
            if (whole) {
                sync_maps();
                // The warps of map m take the m-th half of the rows, of both maps.
#pragma unroll 1
                for (int r0 = m * (RT / 2); r0 < (m + 1) * (RT / 2); r0 += 8) {
                    float u[8], v[8];
                    __syncwarp();
                    tmem_load(tO + r0 + lanes, u);
                    tmem_load(tO + RT + r0 + lanes, v);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        // A row without keys has no sums, not even of NaN.
                        const float f0 = shrink[0][r0 + c], f1 = shrink[1][r0 + c], o = (f0 == 0.f ? 0.f : u[c] * f0) - (f1 == 0.f ? 0.f : v[c] * f1);
                        if (row_out[r0 + c] >= 0 && dv < d.Dv) static_cast<T *>(d.out)[row_out[r0 + c] + dv] = dattn_round<T>(o);
                    }
                }
            } else {
                slot_tile[k] = w.e * d.Hkv + w.n;
                if (!k) slot_last = w.first + w.steps == tile.steps;
                float *to = d.part_o + (slot * RT * 2 + m) * d.Dv + dv;
#pragma unroll 1
                for (int r0 = 0; r0 < used; r0 += 8) {
                    float u[8];
                    __syncwarp();
                    tmem_load(tO + m * RT + r0 + lanes, u);
                    if (dv < d.Dv)
#pragma unroll
                        for (int c = 0; c < 8; ++c) to[(r0 + c) * 2 * d.Dv] = u[c];
                }
            }
            __syncwarp();
            sync_maps();  // the next segment's arrays are the same
        }
        if (threadIdx.x < 2) {
            a.slots[blockIdx.x * 4 + threadIdx.x * 2] = threadIdx.x ? slot_tile[1] : slot_tile[0];
            a.slots[blockIdx.x * 4 + threadIdx.x * 2 + 1] = slot_last;
        }
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        tmem_free(tmem, columns);
    }
    if (threadIdx.x == 0 && *gave_up) atomicOr(&g_paged_gave_up, 1u);
}

// Joins a tile's pieces: the one that begins it is in the second slot of CTA
// blockIdx.x, the others in the first slots of the CTAs after it. A warp per row;
// what it reads depends on two loads before.
constexpr int kJoinRows = 8;

template <typename T> __global__ void __launch_bounds__(32 * kJoinRows) paged_join_kernel(const __grid_constant__ PagedTcArgs a)
{
    const DattnArgs &d = a.d;
    const int c = blockIdx.x, lane = threadIdx.x & 31, v = min(lane * 4, d.Dv - 4), r = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
    if (r >= a.LP * d.G) return;
    pdl_wait();
    const int tile = a.slots[c * 4 + 2];
    int last = lane > 0 && c + lane < a.ctas ? a.slots[(c + lane) * 4 + 1] : 0, pieces = a.ctas - c;
    if (tile < 0) return;
    for (int i = 0; i < a.ctas - c; i += 32) {
        if (i > 0) last = c + i + lane < a.ctas ? a.slots[(c + i + lane) * 4 + 1] : 0;
        const uint32_t any = __ballot_sync(0xffffffffu, last);
        if (any) {
            pieces = i + __ffs(any);
            break;
        }
    }
    const int e = tile / d.Hkv, n = tile - e * d.Hkv, b = e / a.row_tiles, dl = static_cast<int>(d.div_G.div(r));
    const int l = (e - b * a.row_tiles) * a.LP + dl, h = n * d.G + r - dl * d.G;
    if (l >= d.Lq) return;
    const auto slot = [&](int i) { return i == 0 ? static_cast<int64_t>(c) * 2 + 1 : static_cast<int64_t>(c + i) * 2; };
    const auto ml = [&](int i) {  // of both maps
        return i < pieces ? *reinterpret_cast<const float4 *>(d.part_ml + (slot(i) * a.RT + r) * 4) : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    };
    float4 w = ml(lane);
    float top[2] = {w.x, w.z};
    for (int i = lane + 32; i < pieces; i += 32) {
        const float4 x = ml(i);
        top[0] = fmaxf(top[0], x.x);
        top[1] = fmaxf(top[1], x.z);
    }
    for (int m = 0; m < 2; ++m) top[m] = warp_max(top[m]);
    float sum[2] = {0.f, 0.f};
    float4 o[2] = {};
    for (int base = 0; base < pieces; base += 32) {
        if (base > 0) w = ml(base + lane);
        const float f[2] = {ex2(w.x - top[0]), ex2(w.z - top[1])};
        sum[0] = fmaf(w.y, f[0], sum[0]);
        sum[1] = fmaf(w.w, f[1], sum[1]);
        const int here = min(pieces - base, 32);
        // Four pieces at a time, which the loads' latency is spread over; one past
        // the last has a factor of 0 and is read in the last's place.
        for (int i0 = 0; i0 < here; i0 += 4) {
            float4 x[4][2];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    x[k][m] = *reinterpret_cast<const float4 *>(d.part_o + ((slot(min(base + i0 + k, pieces - 1)) * a.RT + r) * 2 + m) * d.Dv + v);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const float g = __shfl_sync(0xffffffffu, f[m], i0 + k), keep = i0 + k < here ? g : 0.f;
                    if (keep == 0.f) continue;  // uniform; what is there may be anything
                    o[m].x = fmaf(x[k][m].x, g, o[m].x);
                    o[m].y = fmaf(x[k][m].y, g, o[m].y);
                    o[m].z = fmaf(x[k][m].z, g, o[m].z);
                    o[m].w = fmaf(x[k][m].w, g, o[m].w);
                }
        }
    }
    for (int m = 0; m < 2; ++m)
        for (int k = 16; k; k >>= 1) sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], k);
    if (lane * 4 >= d.Dv) return;
    const bool live = l < paged_count(d, b);
    const float f0 = sum[0] == 0.f || !live ? 0.f : 1.f / sum[0], f1 = sum[1] == 0.f || !live ? 0.f : d.lam[h] / sum[1];
    const auto out = [&](float x, float y) { return dattn_round<T>((f0 == 0.f ? 0.f : x * f0) - (f1 == 0.f ? 0.f : y * f1)); };
    T *to = static_cast<T *>(d.out) + ((static_cast<int64_t>(b) * d.Lq + l) * d.H + h) * d.Dv + v;
    to[0] = out(o[0].x, o[1].x);
    to[1] = out(o[0].y, o[1].y);
    to[2] = out(o[0].z, o[1].z);
    to[3] = out(o[0].w, o[1].w);
}

template <typename T, int DP, int VP, int RT>
cudaError_t launch_tc(const PagedTcArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st)
{
    using F = PgShared<DP, VP, RT>;
    const size_t smem = F::bytes + 1024 + paged_bias_bytes(a.d.nb, a.d.H, a.d.reach);
    const auto kernel = paged_tc_kernel<T, DP, VP, RT>;
    cudaError_t e = allow_shared(kernel, F::bytes + 1024 + kPgBias);
    if (e != cudaSuccess) return e;
    kernel<<<a.ctas, kPgThreads, smem, st>>>(a, mq, mk, mv);
    e = cudaGetLastError();
    if (e == cudaSuccess && a.ctas > 1 && a.d.Lk > kStep)  // otherwise no tile has pieces
        e = launch_pdl(paged_join_kernel<T>, dim3(a.ctas, (a.LP * a.d.G + kJoinRows - 1) / kJoinRows), dim3(32 * kJoinRows), 0, st, a);
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
