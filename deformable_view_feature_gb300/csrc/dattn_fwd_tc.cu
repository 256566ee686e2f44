// Differential attention forward on the tensor cores (include/dattn.h), for
// bf16 and fp16.
//
// One CTA takes 128 rows (queries x the heads that share a key head) and
// walks over the keys in steps of 64. The two softmax maps take the place of
// the two row tiles by which such a kernel usually keeps its units busy: four
// warps turn the scores of map 0 into weights, four those of map 1, and the
// tensor core meanwhile forms P v and the next scores of either; K is loaded
// once for both scores and V once for both products.
//
// Warps: 0-3 softmax of map 0 and 4-7 of map 1 (a thread per row, so row
// maxima and sums need no exchange), 8 loads by TMA, 9 issues the products,
// 10 prepares each step's positions and masks. Tensor memory: two steps'
// scores of each map, 64 columns, whose first 32 then hold the map's weights
// in 16 bits as the operand of P v, and the two outputs. Steps of 128 keys
// would use the tensor core better, but leave room for one step's scores
// only: the softmax warps then waited 1500 of 3670 clocks for theirs.
// A step now takes 1,470 clocks, 768 of them multiplication; the chain from
// scores to weights to the next products bounds it, not a unit (tensor pipe
// 49 %, exponentials 26 % of their peak). 2 x 8 heads of 8,192 tokens, causal,
// D = 64, Dv = 128: 363 us, 376 with what the backward pass needs, 1.1 PFLOP/s.
// Eight caches of 18,432 to 32,768 keys: 114 us, 3.7 TB/s; each is split into
// four, so that the longest's CTAs walk 128 steps where an even share of all
// steps on 152 SMs would be 84.
// The weights go into their product rounded to the inputs' type: with what the
// rounding took as a second operand the outputs' errors were those of fp32
// weights (bf16 0.0017 for 0.0025, 2-norm), but 8,192 tokens took 440 us and
// the caches 140.
// A thread raises its row's reference, and rescales the row's output, only
// when a step's best score exceeds the one that the reference was made from by
// more than 2^8. In fp16 the reference lies 2^7 below that score: weights of up
// to 2^15 use the type's whole range, and weights round to nothing below 2^-32
// of the best instead of 2^-25. Many keys of 2^-25 each are not nothing together.
#include "dattn_tc.cuh"

namespace da {
namespace {

using namespace tc;

constexpr int kTile = 128;            // rows
constexpr int kKeys = 64;             // keys per step
constexpr int kFwdThreads = 11 * 32;
constexpr float kSlack = 8.f;         // log2 of how far weights may exceed their first best
template <typename T> constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;  // log2 of that best

// What the softmax warps need to know of a step's keys.
struct alignas(16) KeyInfo {
    float bound[kKeys];  // +infinity, or -infinity for a key that is not to be used
    int pos[kKeys];
    int lo, hi;          // smallest and largest position of those used
    uint32_t all;        // every key is to be used
};

template <int DP, int VP> struct FwdShared {
    static constexpr int row = DP * 2;                 // bytes of a row of q or k
    static constexpr int q = kTile * row, k = kKeys * row;  // of one map
    static constexpr int vblock = kKeys * 128;         // of 64 columns of V
    static constexpr int stage = 2 * k + (VP / 64) * vblock;
    static constexpr int stages = 4;
    static constexpr int outputs = kTile * VP * 2;     // of the tile's output, and of each word saved with it
    static constexpr int operands = 2 * q + stages * stage;
    static constexpr int bytes = operands > 4 * outputs ? operands : 4 * outputs;
};

// Floats of the bias of G heads by relative position, with the ends' values
// repeated for a step more on either side.
__host__ __device__ inline int bias_span(int reach) { return 2 * (reach + kKeys) + 1; }

// A barrier's wait names a phase by its parity only, so nobody may lag two
// phases behind: what the tensor core passes up to a step ahead has a barrier
// for even steps and one for odd. A wait costs some 140 clocks even where it
// does not wait, so the warp that issues the products has three to a step:
// `ready` stands for K, V and the step's infos, and s_full for all products
// issued before, P v of two steps before among them.
struct FwdBars {
    uint64_t q_full, fin;
    uint64_t full[4], ready[4], empty[4];   // of a stage: loaded, cleared of unused keys, free
    uint64_t s_full[2][2], p_full[2][2];    // of each map, for even and odd steps
    uint32_t tmem, gave_up;
};

// Device word for waits that ran out (dattn_device_status).
__device__ uint32_t g_gave_up;

template <typename T, int DP, int VP>
__global__ void __launch_bounds__(kFwdThreads, 1)
    dattn_fwd_tc_kernel(const __grid_constant__ DattnArgs a, const __grid_constant__ CUtensorMap mq,
                        const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv)
{
    using F = FwdShared<DP, VP>;
    constexpr int NS = F::stages;
    constexpr bool bf16 = sizeof(T) == 2 && !std::is_same<T, __half>::value;
    extern __shared__ unsigned char raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    __shared__ FwdBars bars;
    __shared__ KeyInfo infos[NS];
    __shared__ float row_l[2][kTile];
    float *table = reinterpret_cast<float *>(base + F::bytes);  // [G][span], times log2(e)

    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int LP = kTile / a.G;  // queries of a tile
    // The tiles with most keys to see first, of all heads and batch items.
    const int bn = blockIdx.x % (a.B * a.Hkv), rest = blockIdx.x / (a.B * a.Hkv);
    const int b = bn / a.Hkv, n = bn - b * a.Hkv, split = rest % a.splits;
    const int l0 = ((a.Lq + LP - 1) / LP - 1 - rest / a.splits) * LP;
    const int len = dattn_length(a, b);
    int end = len;
    // Keys after the tile's last query end the walk where positions are indices.
    const bool indices = !a.pos_q && !a.pos_k;
    if (a.causal && indices) end = min(end, max(len - a.Lq + min(l0 + LP, a.Lq), 0));
    const int per = ((end + kKeys - 1) / kKeys + a.splits - 1) / a.splits * kKeys;
    const int jb = split * per;
    end = min(end, jb + per);
    const int T_ = end > jb ? (end - jb + kKeys - 1) / kKeys : 0;
    const int span = bias_span(a.reach);

    if (threadIdx.x == 0) {
        bar_init(&bars.q_full, 1);
        bar_init(&bars.fin, 1);
        for (int s = 0; s < NS; ++s) {
            bar_init(&bars.full[s], 1);
            bar_init(&bars.ready[s], 1);
            bar_init(&bars.empty[s], 1);
        }
        for (int m = 0; m < 2; ++m)
            for (int i = 0; i < 2; ++i) {
                bar_init(&bars.s_full[m][i], 1);
                bar_init(&bars.p_full[m][i], 4);
            }
        bars.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
    }
    if (warp == 9) tmem_alloc(&bars.tmem, 512);
    for (int i = threadIdx.x; i < a.G * span; i += kFwdThreads) {
        const int g = i / span, rel = min(max(i - g * span - kKeys, 0), 2 * a.reach);
        table[i] = a.nb ? a.table[min(max(a.bmap[rel], 0), a.nb - 1) * a.H + n * a.G + g] * kLog2e : 0.f;
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(bars.tmem);
    volatile uint32_t *gave_up = &bars.gave_up;
    auto tS = [&](int m, int t) { return tmem + m * 128 + (t & 1) * 64; };
    const uint32_t tO[2] = {tmem + 256, tmem + 256 + VP};
    const uint32_t sq = smem_addr(base), sst = sq + 2 * F::q;

    if (warp == 8) {
        if (lane == 0 && T_ > 0) {
            bar_expect(&bars.q_full, 2 * F::row * a.G * LP);
            for (int m = 0; m < 2; ++m) tma_load(&mq, &bars.q_full, base + m * F::q, 0, m, n * a.G, l0, b);
            for (int t = 0; t < T_; ++t) {
                const int s = t % NS;
                unsigned char *st = base + 2 * F::q + s * F::stage;
                bar_wait(&bars.empty[s], ((t / NS) & 1) ^ 1, gave_up);
                bar_expect(&bars.full[s], F::stage);
                for (int m = 0; m < 2; ++m) tma_load(&mk, &bars.full[s], st + m * F::k, 0, m, n, jb + t * kKeys, b);
                for (int c = 0; c < VP / 64; ++c)
                    tma_load(&mv, &bars.full[s], st + 2 * F::k + c * F::vblock, c * 64, 0, n, jb + t * kKeys, b);
            }
            if (*gave_up) {  // leave no copy in flight
                bar_drain(&bars.q_full, 0);
                for (int t = max(0, T_ - NS); t < T_; ++t) bar_drain(&bars.full[t % NS], (t / NS) & 1);
            }
        }
    } else if (warp == 9) {
        if (T_ > 0) {
            // All lanes walk through the steps, one issues: addresses then
            // stay in uniform registers. (Issued from a branch of one lane's
            // own, a product took some 85 clocks and bound the kernel.)
            const bool issue = elect();
            constexpr uint32_t iqk = shape(bf16, kKeys, false), ipv = shape(bf16, VP, true);
            const Operand<F::row> dq = along_row<F::row>(sq), dk = along_row<F::row>(sst);
            const Operand<128> dv = over_rows<128>(sst + 2 * F::k, F::vblock);
            // Scores of map m at step t; past the last, only the notice that
            // the products before are done.
            auto scores = [&](int m, int t) {
                const uint32_t st = (t % NS) * F::stage;
                if (t < T_ && m == 0) bar_wait_warp(&bars.ready[t % NS], (t / NS) & 1, gave_up);
                fence_after();
                if (issue) {
                    if (t < T_)
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i)
                            mma_ss(tS(m, t), dq.at(m * F::q + i * 32), dk.at(st + m * F::k + i * 32), iqk, i > 0);
                    mma_commit(&bars.s_full[m][t & 1]);
                }
                __syncwarp();
            };
            bar_wait_warp(&bars.q_full, 0, gave_up);
#pragma unroll
            for (int i = 0; i < 4; ++i) scores(i & 1, i >> 1);
            for (int t = 0; t < T_; ++t) {
                const int s = t % NS;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    bar_wait_warp(&bars.p_full[m][t & 1], (t >> 1) & 1, gave_up);
                    fence_after();
                    if (issue) {
#pragma unroll
                        for (int i = 0; i < kKeys / 16; ++i)
                            mma_ts(tO[m], tS(m, t) + i * 8, dv.at(s * F::stage + i * 16 * 128), ipv, t > 0 || i > 0);
                        if (m == 1) mma_commit(&bars.empty[s]);
                    }
                    // Into the columns whose weights the products just issued
                    // read: products are formed in the order of their issue.
                    scores(m, t + 2);
                }
            }
            if (issue) mma_commit(&bars.fin);
            bar_drain(&bars.fin, 0);
            __syncwarp();
        }
    } else if (warp == 10) {
        // A step ahead: whether the lane's two keys are to be used, and where
        // they are.
        bool next_use[2];
        int next_pos[2];
        const auto fetch = [&](int t) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int j = jb + t * kKeys + c * 32 + lane;
                const bool in = j < end;
                const int64_t at = static_cast<int64_t>(b) * a.Lk + j;
                next_use[c] = in && (!a.mask || a.mask[at]);
                next_pos[c] = in && a.pos_k ? a.pos_k[at] : j;
            }
        };
        fetch(0);
        for (int t = 0; t < T_; ++t) {
            const int s = t % NS;
            KeyInfo &ki = infos[s];
            const bool use[2] = {next_use[0], next_use[1]};
            const int pos[2] = {next_pos[0], next_pos[1]};
            fetch(t + 1);
            // The stage is free once P v of NS steps ago is done: the softmax
            // warps had by then read its infos, and the products its V.
            bar_wait_warp(&bars.empty[s], ((t / NS) & 1) ^ 1, gave_up);
            int lo = INT32_MAX, hi = INT32_MIN;
            uint32_t every = 0xffffffffu;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                ki.pos[c * 32 + lane] = pos[c];
                ki.bound[c * 32 + lane] = use[c] ? INFINITY : -INFINITY;
                every &= __ballot_sync(0xffffffffu, use[c]);
                if (use[c]) {
                    lo = min(lo, pos[c]);
                    hi = max(hi, pos[c]);
                }
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            if (lane == 0) {
                ki.lo = lo;
                ki.hi = hi;
                ki.all = every == 0xffffffffu;
            }
            bar_wait_warp(&bars.full[s], (t / NS) & 1, gave_up);
            if (every != 0xffffffffu) {
                // 0 * NaN is NaN: the rows of V of unused keys become zeros
                // (past the tensor's end TMA wrote them).
                unsigned char *v = base + 2 * F::q + s * F::stage + 2 * F::k;
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (!use[c] && jb + t * kKeys + c * 32 + lane < a.Lk)
#pragma unroll
                        for (int i = 0; i < VP / 8; ++i)  // neighbouring rows start at different banks
                            *reinterpret_cast<uint4 *>(v + (i / 8) * F::vblock + (c * 32 + lane) * 128 + (((i + lane) & 7) << 4)) =
                                make_uint4(0, 0, 0, 0);
                fence_async();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.ready[s]);
        }
    } else {
        const int m = warp >> 2, rl = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int dl = static_cast<int>(a.div_G.div(rl)), g = rl - dl * a.G, l = l0 + dl;
        const bool live = rl < LP * a.G && l < a.Lq;
        const int pos = !live ? 0 : a.pos_q ? a.pos_q[static_cast<int64_t>(b) * a.Lq + l] : len - a.Lq + l;
        const float *tb = table + g * span + a.reach + kKeys;  // a row past the tile's heads still reads inside the table
        float ref = -INFINITY;
        float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
        for (int t = 0; t < T_; ++t) {
            const KeyInfo &ki = infos[t % NS];
            bar_wait_warp(&bars.s_full[m][t & 1], (t >> 1) & 1, gave_up);
            fence_after();
            float s[kKeys];
            tmem_load(tS(m, t) + lanes, s);
            const int rlo = ki.lo - pos, rhi = ki.hi - pos;
            const bool all = ki.all;
            // One bias for all of the row's keys in this step, none of them later.
            const bool even = !live || (!(a.causal && rhi > 0) && (a.nb == 0 || rlo >= a.reach || rhi <= -a.reach || rlo == rhi));
            const bool fast = __all_sync(0xffffffffu, even) && a.scale_log2 > 0.f;
            float mul = a.scale_log2, add = 0.f;
            if (fast) {
                add = tb[min(max(rlo, -a.reach), a.reach)];
            } else {
                const float mul_all = a.scale_log2;
                if (indices) {
                    // Positions rise by one from key to key: so do places in the table.
                    const int rel = jb + t * kKeys - pos, seen = a.causal ? -rel : kKeys;
                    const float *p = tb + min(max(rel, -a.reach - kKeys), a.reach + 1);
#pragma unroll
                    for (int i = 0; i < kKeys; ++i) {
                        const float x = fmaf(s[i], mul_all, p[i]);
                        s[i] = i <= seen ? x : -INFINITY;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kKeys; ++i) {
                        const int rel = ki.pos[i] - pos;
                        const float x = fmaf(s[i], mul_all, tb[min(max(rel, -a.reach), a.reach)]);
                        s[i] = a.causal && rel > 0 ? -INFINITY : x;
                    }
                }
                mul = 1.f;
            }
            if (!all) {
                // The smaller of a NaN and -infinity is -infinity.
#pragma unroll
                for (int i = 0; i < kKeys; i += 4) {
                    const float4 bound = *reinterpret_cast<const float4 *>(&ki.bound[i]);
                    s[i] = fminf(s[i], bound.x);
                    s[i + 1] = fminf(s[i + 1], bound.y);
                    s[i + 2] = fminf(s[i + 2], bound.z);
                    s[i + 3] = fminf(s[i + 3], bound.w);
                }
            }
            float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int i = 4; i < kKeys - 4; i += 8)
#pragma unroll
                for (int c = 0; c < 4; ++c) top[c] = max3(top[c], s[i + c], s[i + 4 + c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) top[c] = fmaxf(top[c], s[kKeys - 4 + c]);
            const float best = fmaf(max3(fmaxf(top[0], top[1]), top[2], top[3]), mul, add);
            // Each row's reference by its own scores alone; rows past the end
            // hold stale values. (Whether the bias is added before the
            // exponent's product or with it is one choice for a warp's rows, so
            // that a row's last bits can depend on which rows lie beside it.)
            const bool raise = live && best > ref + (kLift<T> + kSlack);
            if (__any_sync(0xffffffffu, raise)) {
                const float next = raise ? best - kLift<T> : ref;
                const float shrink = raise ? ex2(ref - next) : 1.f;
                ref = next;
                const float2 sh = {shrink, shrink};
                sum[0] = mul2(sum[0], sh);
                sum[1] = mul2(sum[1], sh);
                if (t > 0) {
                    // P v of step t - 1 was issued just before the scores of step t + 1.
                    bar_wait_warp(&bars.s_full[m][(t + 1) & 1], ((t + 1) >> 1) & 1, gave_up);
                    fence_after();
#pragma unroll 1
                    for (int c = 0; c < VP; c += 32) {
                        float o[32];
                        tmem_load(tO[m] + lanes + c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= shrink;
                        tmem_store(tO[m] + lanes + c, o);
                    }
                }
            }
            const float off = add - (ref == -INFINITY ? 0.f : ref);
            const float2 mul_2 = {mul, mul}, off_2 = {off, off};
            uint32_t p[kKeys / 2];
#pragma unroll
            for (int i = 0; i < kKeys / 2; ++i) {
                float2 x = fma2({s[2 * i], s[2 * i + 1]}, mul_2, off_2);
                x.x = ex2(x.x);
                x.y = ex2(x.y);
                sum[i & 1] = add2(sum[i & 1], x);
                p[i] = pack2<T>(x.x, x.y);
            }
            tmem_store(tS(m, t) + lanes, p);
            tmem_store_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.p_full[m][t & 1]);
        }
        row_l[m][rl] = sum[0].x + sum[0].y + (sum[1].x + sum[1].y);
        if (T_ > 0) bar_wait_warp(&bars.fin, 0, gave_up);
        fence_after();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float s0 = row_l[0][rl], s1 = row_l[1][rl];
        const float w0 = s0 == 0.f ? 0.f : 1.f / s0, w1 = s1 == 0.f ? 0.f : 1.f / s1;
        const int h = n * a.G + (live ? g : 0);
        const float nan = *gave_up ? NAN : 0.f;
        const float lam = a.lam[h];
        const int64_t pt = ((static_cast<int64_t>(b) * a.Hkv + n) * a.rows + static_cast<int64_t>(l) * a.G + g) * a.splits + split;
        // Outputs go through shared memory, which the products have left, so
        // that neighbouring lanes store neighbouring pieces: piece p of row r
        // of word k lies at piece p ^ (r % 8).
        const auto cell = [&](int k, int r, int p) { return reinterpret_cast<uint4 *>(base + k * F::outputs + r * VP * 2 + ((p ^ (r & 7)) << 4)); };
        // The warps of map m take the m-th half of the columns.
#pragma unroll 1
        for (int c = m * (VP / 2); c < (m + 1) * (VP / 2); c += 32) {
            float x[32], y[32];
            __syncwarp();
            if (T_ > 0) {
                tmem_load(tO[0] + lanes + c, x);
                tmem_load(tO[1] + lanes + c, y);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = y[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                if (!live || c + i >= a.Dv) continue;
                if (a.splits > 1) {
                    float *o = a.part_o + pt * 2 * a.Dv + c + i;
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        *reinterpret_cast<float4 *>(o + e) = make_float4(x[i + e], x[i + e + 1], x[i + e + 2], x[i + e + 3]);
                        *reinterpret_cast<float4 *>(o + a.Dv + e) = make_float4(y[i + e], y[i + e + 1], y[i + e + 2], y[i + e + 3]);
                    }
                    continue;
                }
                const int p = (c + i) / 8;
                uint32_t u[4], w[4], ru[4], rw[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y0 = y[i + 2 * e] * w1, y1 = y[i + 2 * e + 1] * w1;
                    const float x0 = fmaf(-lam, y0, x[i + 2 * e] * w0), x1 = fmaf(-lam, y1, x[i + 2 * e + 1] * w0);
                    u[e] = pack2<T>(x0, x1);
                    if (!a.out1) continue;
                    w[e] = pack2<T>(y0, y1);
                    ru[e] = rest2<T>(u[e], x0, x1);
                    rw[e] = rest2<T>(w[e], y0, y1);
                }
                *cell(0, rl, p) = make_uint4(u[0], u[1], u[2], u[3]);
                if (!a.out1) continue;
                *cell(1, rl, p) = make_uint4(ru[0], ru[1], ru[2], ru[3]);
                *cell(2, rl, p) = make_uint4(w[0], w[1], w[2], w[3]);
                *cell(3, rl, p) = make_uint4(rw[0], rw[1], rw[2], rw[3]);
            }
        }
        if (a.splits == 1) {
            asm volatile("bar.sync 1, 256;" ::: "memory");
            constexpr int P = VP / 8, passes = kTile * P / 256;
            const bool wide = aligned16(a.out) && aligned16(a.out1), bad = *gave_up;
            const int p = threadIdx.x % P, r0 = threadIdx.x / P, words = a.out1 ? 1 + kSaved<T> : 1;
            int64_t at[passes];  // of the thread's rows, or -1
#pragma unroll
            for (int i = 0; i < passes; ++i) {
                const int r = r0 + i * (256 / P), dr = static_cast<int>(a.div_G.div(r));
                at[i] = dr >= LP || l0 + dr >= a.Lq || p * 8 >= a.Dv
                            ? -1
                            : ((static_cast<int64_t>(b) * a.Lq + l0 + dr) * a.H + n * a.G + r - dr * a.G) * a.Dv;
            }
#pragma unroll 1
            for (int k = 0; k < words; ++k) {
                T *to = k == 0 ? static_cast<T *>(a.out) + p * 8 : static_cast<T *>(a.out1) + (k - 1) * a.Dv + p * 8;
                uint4 v[passes];
#pragma unroll
                for (int i = 0; i < passes; ++i) v[i] = *cell(k, r0 + i * (256 / P), p);
#pragma unroll
                for (int i = 0; i < passes; ++i) {
                    if (at[i] < 0) continue;
                    if (bad) v[i] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);  // NaN of either type
                    T *o = to + at[i] * (k == 0 ? 1 : kSaved<T>);
                    if (wide) {
                        *reinterpret_cast<uint4 *>(o) = v[i];
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = reinterpret_cast<const T *>(&v[i])[e];
                    }
                }
            }
        }
        __syncwarp();
        if (live) {
            const float s = row_l[m][rl];
            if (a.splits > 1) {
                a.part_ml[(pt * 2 + m) * 2] = ref;
                a.part_ml[(pt * 2 + m) * 2 + 1] = s + nan;
            } else if (a.lse) {
                a.lse[((static_cast<int64_t>(b) * a.H + h) * 2 + m) * a.Lq + l] = (s == 0.f ? INFINITY : ref + log2f(s)) + nan;
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        tmem_free(tmem, 512);
    }
    if (threadIdx.x == 0 && *gave_up) atomicOr(&g_gave_up, 1u);
}

template <typename T, int DP, int VP>
cudaError_t launch_fwd(const DattnArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st)
{
    using F = FwdShared<DP, VP>;
    const size_t smem = F::bytes + 1024 + sizeof(float) * a.G * bias_span(a.reach);
    const auto kernel = dattn_fwd_tc_kernel<T, DP, VP>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int LP = kTile / a.G;
    const unsigned grid = static_cast<unsigned>((a.Lq + LP - 1) / LP * a.splits) * a.Hkv * a.B;
    kernel<<<grid, kFwdThreads, smem, st>>>(a, mq, mk, mv);
    return cudaGetLastError();
}

template <typename T> cudaError_t fwd_widths(const DattnArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st)
{
    if (a.D <= 32) return a.Dv <= 64 ? launch_fwd<T, 32, 64>(a, mq, mk, mv, st) : launch_fwd<T, 32, 128>(a, mq, mk, mv, st);
    return a.Dv <= 64 ? launch_fwd<T, 64, 64>(a, mq, mk, mv, st) : launch_fwd<T, 64, 128>(a, mq, mk, mv, st);
}

}  // namespace

uint32_t *dattn_gave_up_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_gave_up) == cudaSuccess ? static_cast<uint32_t *>(p) : nullptr;
}

da_status dattn_forward_tensor(const DattnArgs &a, int dtype, cudaStream_t st)
{
    const int wide = a.D <= 32 ? 32 : 64, LP = kTile / a.G;
    CUtensorMap mq, mk, mv;
    da_status e = tensor_map(mq, dtype, a.q, a.D, 2, a.H, a.Lq, a.B, a.qs[3], a.qs[2], a.qs[1], a.qs[0], wide, a.G, LP);
    if (e == DA_OK) e = tensor_map(mk, dtype, a.k, a.D, 2, a.Hkv, a.Lk, a.B, a.ks[3], a.ks[2], a.ks[1], a.ks[0], wide, 1, kKeys);
    if (e == DA_OK) e = tensor_map(mv, dtype, a.v, a.Dv, 1, a.Hkv, a.Lk, a.B, 0, a.vs[2], a.vs[1], a.vs[0], 64, 1, kKeys);
    if (e != DA_OK) return e;
    const cudaError_t c = dtype == DA_BF16 ? fwd_widths<__nv_bfloat16>(a, mq, mk, mv, st) : fwd_widths<__half>(a, mq, mk, mv, st);
    return c == cudaSuccess ? DA_OK : cuda_fail(c, "differential attention launch");
}

}  // namespace da
