// Differential attention backward on the tensor cores (include/dattn.h), for
// bf16 and fp16.
//
// Two kernels, each of which forms the scores again from q, k and the saved
// log-sums. The first owns 128 rows and walks over the keys in tiles of 64:
// grad_q, and the d_m in full fp32 precision (it begins with those of the
// saved outputs, which hold two words a value). The second owns 128 keys and
// walks over the queries of every head that shares them in tiles of 64:
// grad_k, grad_v and the bias table's gradient. Forming e and the scores twice
// costs 28 D products per pair in place of 20 D, but no sum then crosses CTAs:
// no fp32 image of grad_q, no atomics, the same bits in every run.
//
// Since e = g v^T serves both maps, and P_0 - lam P_1 is formed before its
// product with g, a pair costs three products forward and three (grad_k twice,
// grad_v) or two (grad_q twice) back. All products sum in tensor memory.
// With 64 columns a product reads its operands from shared memory for 48
// clocks and multiplies for 32, so the operands that stay lie in tensor memory
// too, as far as it goes: q, g and s_m of the rows in the first kernel, s_m
// in the second, and v and the weights unless Dv is above 64.
//
// At 2 x 8 heads of 8,192 tokens, causal, D = 64, Dv = 128: 476 us for the
// first kernel and 737 for the second, 1,710 and 2,880 clocks a step for 768
// and 1,024 of multiplication. All compute warps work on one step, so its
// phases (scores to registers, exponentials, operands back) do not overlap each
// other, only the products; tensor memory has no room for a second step.
//
// Warps: 0-7 compute (two threads per row or key, each with half of a step's
// 64 columns of both maps), 8 loads by TMA, 9 issues the products, 10 prepares
// positions, masks and per-query values. The scores of step t+1 are formed as
// soon as the compute warps hold those of step t in registers.
#include "dattn_tc.cuh"

namespace da {
namespace {

using namespace tc;

constexpr int kOwn = 128;   // rows or keys that a CTA owns
constexpr int kStep = 64;   // keys or queries of a step
constexpr int kBwdThreads = 11 * 32;
constexpr int kBlock = 128; // bytes of a row of 64 columns

__device__ uint32_t g_gave_up_backward;

template <typename T> constexpr bool is_bf16 = !std::is_same<T, __half>::value;

// fp16 operands need scales of their own: s_m is about a gradient over a
// number of keys, far below the type's normal numbers or, times g v, past its
// largest. |s_m| <= P |e - d| and |e|, |d| <= sum |g| max |v|, so with
//   bound = 2 sum_c |g_c| max(1, |lam|) max |v|
// a power of two brings s_m to at most 2^15: of each row in the first kernel,
// of all rows of the key head in the second, where one sum goes over them. It
// enters with e and d, in the place of their difference's addition, and is
// taken out of the sums in fp32. The weights are formed 2^15 / (1 + max |lam|)
// higher by the exponent. bf16 has fp32's exponents and needs none of it.
template <typename T> constexpr bool kScaled = std::is_same<T, __half>::value;

// The power of two that takes values of up to `bound` to at most 2^15.
__device__ __forceinline__ float scale_to_range(float bound)
{
    if (!(bound > 0.f && bound < INFINITY)) return 1.f;  // nothing to scale, or nothing that would help
    const int e = 14 - (static_cast<int>(__float_as_uint(bound) >> 23) - 127);  // bound < 2^(15 - e)
    return __uint_as_float(static_cast<uint32_t>(min(max(e, -100), 100) + 127) << 23);
}

// Largest |v| of each batch item and key head, over the keys to be used.
constexpr int kMostKeys = 128;  // keys of a CTA
__global__ void __launch_bounds__(256) dattn_most_v_kernel(const __grid_constant__ DattnArgs a)
{
    const int bn = blockIdx.x % (a.B * a.Hkv), b = bn / a.Hkv, n = bn - b * a.Hkv, j0 = blockIdx.x / (a.B * a.Hkv) * kMostKeys;
    const int piece = threadIdx.x & 15;  // of 8 channels
    const int len = dattn_length(a, b);
    const __half *v = static_cast<const __half *>(a.v) + b * a.vs[0] + n * a.vs[2] + piece * 8;
    uint32_t most = 0;  // bits of |v|, in fp16: they order as the values do
#pragma unroll
    for (int i = 0; i < kMostKeys; i += 16) {
        const int j = j0 + i + static_cast<int>(threadIdx.x >> 4);
        if (j >= len || piece * 8 >= a.Dv || (a.mask && !a.mask[static_cast<int64_t>(b) * a.Lk + j])) continue;
        const uint4 u = *reinterpret_cast<const uint4 *>(v + j * a.vs[1]);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) most = __vmaxu2(most, w[c] & 0x7fff7fffu);
    }
    most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
    if ((threadIdx.x & 31) == 0) atomicMax(a.most + bn, __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(most)))));
}

// 32 columns of one row of a [128][64] operand of 16 bits, swizzled as TMA
// would: 16-byte piece i of row r lies at piece i ^ (r % 8).
__device__ __forceinline__ void store_operand(unsigned char *tile, int row, int half, const uint32_t (&p)[16])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(tile + row * kBlock + (((half * 4 + i) ^ (row & 7)) << 4)) =
            make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
}

// 32 columns from `half` on of row `row` of a tile with rows of ROW bytes, to
// 16 columns of tensor memory (two elements each).
template <int ROW> __device__ __forceinline__ void operand_to_tmem(uint32_t addr, const unsigned char *tile, int row, int half)
{
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // 64-byte rows lie two to a swizzled line of 128 bytes.
        const int piece = ROW == 128 ? (half * 4 + i) ^ (row & 7) : i ^ ((row >> 1) & 3);
        const uint4 u = *reinterpret_cast<const uint4 *>(tile + row * ROW + (piece << 4));
        p[4 * i] = u.x;
        p[4 * i + 1] = u.y;
        p[4 * i + 2] = u.z;
        p[4 * i + 3] = u.w;
    }
    tmem_store(addr, p);
}

// Zeroes row r of a tile of queries or keys, two maps of 2 DP bytes and VP / 64
// blocks of 128, by one lane; neighbouring rows start at different banks.
template <int DP, int VP>
__device__ __forceinline__ void clear_key(unsigned char *tile, int row, int map, int blocks, int block)
{
    constexpr int pieces = DP / 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * pieces; ++i)
        *reinterpret_cast<uint4 *>(tile + (i / pieces) * map + row * DP * 2 + (((i + row) & (pieces - 1)) << 4)) = zero;
#pragma unroll
    for (int i = 0; i < VP / 8; ++i)
        *reinterpret_cast<uint4 *>(tile + blocks + (i / 8) * block + row * kBlock + (((i + row) & 7) << 4)) = zero;
}

// A row of 32 values times `f`, rounded, `count` of them from column c.
template <typename T> __device__ __forceinline__ void store_row(T *dst, const float (&x)[32], float f, int count, bool wide)
{
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        if (i >= count) continue;
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = pack2<T>(x[i + 2 * e] * f, x[i + 2 * e + 1] * f);
        if (wide) {
            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[i + e] = reinterpret_cast<const T *>(u)[e];
        }
    }
}

// ---- grad_q ----------------------------------------------------------------

template <int DP, int VP> struct GradQShared {
    static constexpr int row = DP * 2;
    static constexpr int q = kOwn * row, g = kOwn * kBlock;       // one map, one block of 64 columns
    static constexpr int k = kStep * row, v = kStep * kBlock;
    static constexpr int stage = 2 * k + (VP / 64) * v;
    static constexpr int stages = 4;
    static constexpr int at_g = 2 * q, at_stage = at_g + (VP / 64) * g, bytes = at_stage + stages * stage;
    // Columns of tensor memory: two score tiles and e, grad_q, then q, g, s_m.
    static constexpr int c_out = 3 * kStep, c_q = c_out + 2 * DP, c_g = c_q + DP, c_s = c_g + VP / 2;
    static_assert(c_s + kStep <= 512, "tensor memory");
};

struct alignas(16) QKeyInfo {
    float bound[kStep];  // +infinity, or -infinity for a key that is not to be used
    int pos[kStep];
    int lo, hi;          // smallest and largest position of those used
    uint32_t all;        // every key is to be used
};

struct QBars {
    uint64_t q_full, q_ready, fin, s_full, s_free, ds_full;
    uint64_t full[4], empty[4], ready[4];  // of a stage: loaded, free, cleared of unused keys
    uint32_t tmem, gave_up;
};

template <typename T, int DP, int VP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    dattn_grad_q_tc_kernel(const __grid_constant__ DattnArgs a, const __grid_constant__ CUtensorMap mq,
                           const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                           const __grid_constant__ CUtensorMap mg)
{
    using F = GradQShared<DP, VP>;
    constexpr int NS = F::stages;
    extern __shared__ unsigned char raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    __shared__ QBars bars;
    __shared__ QKeyInfo infos[NS];
    __shared__ float part[2][2][kOwn];
    __shared__ int used[2];  // first and last step with a key to be used
    float *table = reinterpret_cast<float *>(base + F::bytes);

    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int LP = kOwn / a.G;
    // The tiles with most keys to see first, of all heads and batch items.
    const int bn = blockIdx.x % (a.B * a.Hkv), b = bn / a.Hkv, n = bn - b * a.Hkv;
    const int l0 = ((a.Lq + LP - 1) / LP - 1 - blockIdx.x / (a.B * a.Hkv)) * LP;
    const int len = dattn_length(a, b);
    int end = len;
    const bool steps_down = a.causal && !a.pos_q && !a.pos_k;  // a query sees the keys up to its own index
    if (steps_down) end = min(end, max(len - a.Lq + min(l0 + LP, a.Lq), 0));
    const int span = 2 * a.reach + 1;

    if (threadIdx.x == 0) {
        bar_init(&bars.q_full, 1);
        bar_init(&bars.q_ready, 8);
        bar_init(&bars.fin, 1);
        bar_init(&bars.s_full, 1);
        bar_init(&bars.s_free, 8);
        bar_init(&bars.ds_full, 8);
        for (int s = 0; s < NS; ++s) {
            bar_init(&bars.full[s], 1);
            bar_init(&bars.empty[s], 1);
            bar_init(&bars.ready[s], 1);
        }
        bars.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
        tma_prefetch(&mg);
    }
    if (warp == 9) tmem_alloc(&bars.tmem, 512);
    if (a.mask && (warp == 8 || warp == 10)) {
        // From the first key on, or from the last one back, 256 at a time.
        const uint8_t *mask = a.mask + static_cast<int64_t>(b) * a.Lk;
        int step = warp == 8 ? 0 : -1;  // without any: none from 0 to -1
        for (int i = 0; i * 256 < end; ++i) {
            const int j = (warp == 8 ? i : (end - 1) / 256 - i) * 256 + lane * 8;
            bool any = false;
#pragma unroll
            for (int c = 0; c < 8; ++c) any |= j + c < end && mask[j + c];
            const uint32_t hit = __ballot_sync(0xffffffffu, any);
            if (hit) {
                step = (j - lane * 8 + (warp == 8 ? __ffs(hit) - 1 : 31 - __clz(hit)) * 8) / kStep;
                break;
            }
        }
        if (lane == 0) used[warp == 10] = step;
    }
    if (a.nb)
        for (int i = threadIdx.x; i < a.G * span; i += kBwdThreads) {
            const int g = i / span, bucket = min(max(a.bmap[i - g * span], 0), a.nb - 1);
            table[i] = a.table[bucket * a.H + n * a.G + g] * kLog2e;
        }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(bars.tmem);
    volatile uint32_t *gave_up = &bars.gave_up;
    // The walk: from key jb on, T_ steps.
    const int jb = a.mask ? used[0] * kStep : 0, T_ = a.mask ? used[1] - used[0] + 1 : (end + kStep - 1) / kStep;
    auto tS = [&](int which) { return tmem + which * kStep; };
    auto tQ = [&](int m) { return tmem + F::c_out + m * DP; };
    const uint32_t sbase = smem_addr(base);

    if (warp == 8) {
        if (lane == 0 && T_ > 0) {
            bar_expect(&bars.q_full, 2 * F::row * a.G * LP + (VP / 64) * kBlock * a.G * LP);
            for (int m = 0; m < 2; ++m) tma_load(&mq, &bars.q_full, base + m * F::q, 0, m, n * a.G, l0, b);
            for (int c = 0; c < VP / 64; ++c) tma_load(&mg, &bars.q_full, base + F::at_g + c * F::g, c * 64, 0, n * a.G, l0, b);
            for (int t = 0; t < T_; ++t) {
                const int s = t % NS;
                unsigned char *st = base + F::at_stage + s * F::stage;
                bar_wait(&bars.empty[s], ((t / NS) & 1) ^ 1, gave_up);
                bar_expect(&bars.full[s], F::stage);
                for (int m = 0; m < 2; ++m) tma_load(&mk, &bars.full[s], st + m * F::k, 0, m, n, jb + t * kStep, b);
                for (int c = 0; c < VP / 64; ++c)
                    tma_load(&mv, &bars.full[s], st + 2 * F::k + c * F::v, c * 64, 0, n, jb + t * kStep, b);
            }
            if (*gave_up) {
                bar_drain(&bars.q_full, 0);
                for (int t = max(0, T_ - NS); t < T_; ++t) bar_drain(&bars.full[t % NS], (t / NS) & 1);
            }
        }
    } else if (warp == 9) {
        if (T_ > 0) {
            const bool issue = elect();
            constexpr uint32_t is = shape(is_bf16<T>, kStep, false), iq = shape(is_bf16<T>, DP, true);
            const Operand<F::row> dk = along_row<F::row>(sbase + F::at_stage), dkr = over_rows<F::row>(sbase + F::at_stage, F::k);
            const Operand<128> dv = along_row<128>(sbase + F::at_stage + 2 * F::k);
            auto scores = [&](int t) {
                const uint32_t st = (t % NS) * F::stage;
                bar_wait_warp(&bars.ready[t % NS], (t / NS) & 1, gave_up);
                if (t > 0) bar_wait_warp(&bars.s_free, (t - 1) & 1, gave_up);
                fence_after();
                if (issue) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i)
                            mma_ts(tS(m), tmem + F::c_q + m * (DP / 2) + i * 8, dk.at(st + m * F::k + i * 32), is, i > 0);
#pragma unroll
                    for (int i = 0; i < VP / 16; ++i)
                        mma_ts(tS(2), tmem + F::c_g + i * 8, dv.at(st + (i / 4) * F::v + (i % 4) * 32), is, i > 0);
                    mma_commit(&bars.s_full);
                }
                __syncwarp();
            };
            bar_wait_warp(&bars.q_ready, 0, gave_up);
            scores(0);
            for (int t = 0; t < T_; ++t) {
                if (t + 1 < T_) scores(t + 1);
                bar_wait_warp(&bars.ds_full, t & 1, gave_up);
                fence_after();
                if (issue) {
                    const uint32_t st = (t % NS) * F::stage;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < kStep / 16; ++i)
                            mma_ts(tQ(m), tmem + F::c_s + m * (kStep / 2) + i * 8, dkr.at(st + m * F::k + i * 16 * F::row), iq, t > 0 || i > 0);
                    mma_commit(&bars.empty[t % NS]);
                }
                __syncwarp();
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
                const int j = jb + t * kStep + c * 32 + lane;
                const bool in = j < end;
                const int64_t at = static_cast<int64_t>(b) * a.Lk + j;
                next_use[c] = in && (!a.mask || a.mask[at]);
                next_pos[c] = in && a.pos_k ? a.pos_k[at] : j;
            }
        };
        fetch(0);
        for (int t = 0; t < T_; ++t) {
            const int s = t % NS;
            QKeyInfo &ki = infos[s];
            const bool use[2] = {next_use[0], next_use[1]};
            const int pos[2] = {next_pos[0], next_pos[1]};
            fetch(t + 1);
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
                // Unused keys (past the tensor's end TMA wrote zeros): 0 * NaN
                // in s k and e would be NaN.
                unsigned char *st = base + F::at_stage + s * F::stage;
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (!use[c] && jb + t * kStep + c * 32 + lane < a.Lk) clear_key<DP, VP>(st, c * 32 + lane, F::k, 2 * F::k, F::v);
                fence_async();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.ready[s]);
        }
    } else {
        const int half = warp >> 2, rl = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int dl = static_cast<int>(a.div_G.div(rl)), g = rl - dl * a.G, l = l0 + dl;
        const bool live = rl < LP * a.G && l < a.Lq;
        const int h = n * a.G + (live ? g : 0);
        const int pos = !live ? 0 : a.pos_q ? a.pos_q[static_cast<int64_t>(b) * a.Lq + l] : len - a.Lq + l;
        const float *tb = table + g * span + a.reach;
        const float lam = a.lam[h], nlam = -lam;
        float lse[2] = {INFINITY, INFINITY}, d[2];
        if (live)
            for (int m = 0; m < 2; ++m) lse[m] = a.lse[((static_cast<int64_t>(b) * a.H + h) * 2 + m) * a.Lq + l];
        // g times the saved outputs: a row's pieces by neighbouring lanes.
        constexpr int P = VP / 8;
        const int piece = threadIdx.x % P;
#pragma unroll 4
        for (int r = threadIdx.x / P; r < kOwn; r += 256 / P) {
            const int dr = static_cast<int>(a.div_G.div(r)), of = r - dr * a.G;
            float d0 = 0.f, d1 = 0.f, sum = 0.f;  // the last of |g|
            if (dr < LP && l0 + dr < a.Lq && piece * 8 < a.Dv) {
                const int64_t row = (static_cast<int64_t>(b) * a.Lq + l0 + dr) * a.H + n * a.G + of;
                const auto eight = [](const void *p, int64_t at) { return *reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + at); };
                const int64_t at = row * a.Dv + piece * 8, save = row * kSaved<T> * a.Dv + piece * 8;
                const uint4 ug = eight(a.grad_out, at), uo = eight(a.out, at), ur = eight(a.out1, save), u1 = eight(a.out1, save + a.Dv),
                            u1r = eight(a.out1, save + 2 * a.Dv);
                const T *vg = reinterpret_cast<const T *>(&ug), *vo = reinterpret_cast<const T *>(&uo), *vr = reinterpret_cast<const T *>(&ur),
                        *v1 = reinterpret_cast<const T *>(&u1), *v1r = reinterpret_cast<const T *>(&u1r);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    d0 = fmaf(dattn_float(vg[e]), dattn_whole(vo[e], vr[e]), d0);
                    d1 = fmaf(dattn_float(vg[e]), dattn_whole(v1[e], v1r[e]), d1);
                    if (kScaled<T>) sum += fabsf(dattn_float(vg[e]));
                }
            }
#pragma unroll
            for (int o = P / 2; o; o >>= 1) {
                d0 += __shfl_xor_sync(0xffffffffu, d0, o);
                d1 += __shfl_xor_sync(0xffffffffu, d1, o);
                if (kScaled<T>) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            if (piece == 0) {
                part[0][0][r] = d0;
                part[1][0][r] = d1;
                if (kScaled<T>) part[0][1][r] = sum;
            }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        d[1] = part[1][0][rl];
        d[0] = fmaf(lam, d[1], part[0][0][rl]);  // out = o_0 - lam o_1
        const bool none = lse[0] == INFINITY;  // sees no key: whatever g holds there is not used
        if (none) d[0] = d[1] = 0.f;
        float f = 1.f;  // s_m is formed times f
        if (kScaled<T>) {
            const float of_g = none ? 0.f : 2.f * part[0][1][rl] * fmaxf(1.f, fabsf(lam));
            f = scale_to_range(of_g * __uint_as_float(a.most[bn]));
            const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(of_g));
            if (half == 0 && lane == 0) atomicMax(a.most + a.B * a.Hkv + bn, most);
        }
        if (T_ > 0) {  // the rows' operands to tensor memory
            bar_wait_warp(&bars.q_full, 0, gave_up);
            for (int m = 0; m < 2; ++m)
                if (DP == 64 || half == m)
                    operand_to_tmem<F::row>(tmem + F::c_q + m * (DP / 2) + (DP == 64 ? half * 16 : 0) + lanes, base + m * F::q, rl, half);
            for (int c = 0; c < VP / 64; ++c)
                operand_to_tmem<128>(tmem + F::c_g + c * 32 + half * 16 + lanes, base + F::at_g + c * F::g, rl, half);
            tmem_store_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.q_ready);
        }
        const float2 nd[2] = {{-d[0] * f, -d[0] * f}, {-d[1] * f, -d[1] * f}}, f_2 = {f, f};
        const auto less_d = [&](float2 e, int m) { return kScaled<T> ? fma2(e, f_2, nd[m]) : add2(e, nd[m]); };
        float2 rest[2] = {{0.f, 0.f}, {0.f, 0.f}};
        // Whether the first step holds all keys that the row sees, or that some row of the tile does.
        const bool whole = T_ == 1 || (steps_down && pos < jb + kStep), some = T_ == 1 || (steps_down && len - a.Lq + l0 < jb + kStep);
        // A step, by_itself the first one where whole rows take d_m from it (in
        // one loop with the others it cost every step, 1 % at 8,192 tokens).
        const auto step = [&](int t, auto by_itself) {
            const QKeyInfo &ki = infos[t % NS];
            bar_wait_warp(&bars.s_full, t & 1, gave_up);
            fence_after();
            float e[32], x[2][32];
            tmem_load3(tS(2) + lanes + half * 32, tS(0) + lanes + half * 32, tS(1) + lanes + half * 32, e, x[0], x[1]);
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.s_free);
            const int rlo = ki.lo - pos, rhi = ki.hi - pos;
            const bool all = ki.all;
            const bool even = !live || (!none && !(a.causal && rhi > 0) &&
                                        (a.nb == 0 || rlo >= a.reach || rhi <= -a.reach || rlo == rhi));
            const bool fast = __all_sync(0xffffffffu, even) && a.scale_log2 > 0.f;
            const float bias_all = a.nb ? tb[min(max(rlo, -a.reach), a.reach)] : 0.f;
            float add[2] = {-lse[0], -lse[1]}, mul = a.scale_log2;
            if (fast) {
                add[0] += bias_all;
                add[1] += bias_all;
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int rel = ki.pos[half * 32 + i] - pos;
                    const float bias = a.nb ? tb[min(max(rel, -a.reach), a.reach)] : 0.f;
                    const bool on = !(a.causal && rel > 0) && !none;
                    x[0][i] = on ? fmaf(x[0][i], mul, bias + add[0]) : -INFINITY;
                    x[1][i] = on ? fmaf(x[1][i], mul, bias + add[1]) : -INFINITY;
                }
                mul = 1.f;
                add[0] = add[1] = 0.f;
            }
            if (!all) {
                // The smaller of a NaN and -infinity is -infinity; e is 0 there.
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 bound = *reinterpret_cast<const float4 *>(&ki.bound[half * 32 + i]);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        x[m][i] = fminf(x[m][i], bound.x);
                        x[m][i + 1] = fminf(x[m][i + 1], bound.y);
                        x[m][i + 2] = fminf(x[m][i + 2], bound.z);
                        x[m][i + 3] = fminf(x[m][i + 3], bound.w);
                    }
                }
            }
            uint32_t p[2][16];
            const float2 mul_2 = {mul, mul}, a0 = {add[0], add[0]}, a1 = {add[1], add[1]}, nl = {nlam, nlam};
            if constexpr (by_itself.value) {
                // All of a whole row's keys are here: weights that sum to 1 and
                // d_m from them, so that a row of one key gives exactly 0.
                float y[2] = {0.f, 0.f};
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float z = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        x[m][i] = none ? 0.f : ex2(fmaf(x[m][i], mul, add[m]));
                        z += x[m][i];
                    }
                    part[m][half][rl] = z;
                }
                asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const float z = whole ? part[m][0][rl] + part[m][1][rl] : 1.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        x[m][i] = none ? 0.f : x[m][i] / z;
                        e[i] = none ? 0.f : e[i];
                        y[m] = fmaf(x[m][i], e[i], y[m]);
                    }
                }
                asm volatile("bar.sync 1, 256;" ::: "memory");
                part[0][half][rl] = y[0];
                part[1][half][rl] = y[1];
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (whole)
                    for (int m = 0; m < 2; ++m) d[m] = part[m][0][rl] + part[m][1][rl];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float s[2][2];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int k = 0; k < 2; ++k) s[m][k] = x[m][2 * i + k] * ((e[2 * i + k] - d[m]) * f);
                    rest[0] = add2(rest[0], {s[0][0], s[0][1]});
                    rest[1] = add2(rest[1], {s[1][0], s[1][1]});
                    p[0][i] = pack2<T>(s[0][0], s[0][1]);
                    p[1][i] = pack2<T>(nlam * s[1][0], nlam * s[1][1]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 ei = {none ? 0.f : e[2 * i], none ? 0.f : e[2 * i + 1]};
                    float2 w0 = fma2({x[0][2 * i], x[0][2 * i + 1]}, mul_2, a0), w1 = fma2({x[1][2 * i], x[1][2 * i + 1]}, mul_2, a1);
                    w0.x = ex2(w0.x);
                    w0.y = ex2(w0.y);
                    w1.x = ex2(w1.x);
                    w1.y = ex2(w1.y);
                    const float2 s0 = mul2(w0, less_d(ei, 0)), s1 = mul2(w1, less_d(ei, 1));
                    rest[0] = add2(rest[0], s0);
                    rest[1] = add2(rest[1], s1);
                    const float2 s1l = mul2(s1, nl);
                    p[0][i] = pack2<T>(s0.x, s0.y);
                    p[1][i] = pack2<T>(s1l.x, s1l.y);
                }
            }
            if (t > 0) bar_wait_warp(&bars.empty[(t - 1) % NS], ((t - 1) / NS) & 1, gave_up);  // s_m of step t - 1 was used
            tmem_store(tmem + F::c_s + half * 16 + lanes, p[0]);
            tmem_store(tmem + F::c_s + kStep / 2 + half * 16 + lanes, p[1]);
            tmem_store_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.ds_full);
        };
        int t = 0;
        if (T_ > 0 && some) step(t++, std::true_type{});
        for (; t < T_; ++t) step(t, std::false_type{});
        asm volatile("bar.sync 1, 256;" ::: "memory");
        for (int m = 0; m < 2; ++m) part[m][half][rl] = rest[m].x + rest[m].y;
        if (T_ > 0) bar_wait(&bars.fin, 0, gave_up);
        fence_after();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const int m = half;  // the warps of each half write one map
        const float nan = *gave_up ? NAN : 0.f;
        if (live)
            a.delta[((static_cast<int64_t>(b) * a.Hkv + n) * 2 + m) * a.rows + static_cast<int64_t>(l) * a.G + g] =
                (none ? 0.f : d[m] + (part[m][0][rl] + part[m][1][rl]) / f) + nan;
        T *dst = static_cast<T *>(a.grad_q) + (((static_cast<int64_t>(b) * a.Lq + l) * a.H + h) * 2 + m) * a.D;
        const bool wide = aligned16(a.grad_q);
#pragma unroll 1
        for (int c = 0; c < DP; c += 32) {
            float x[32];
            __syncwarp();
            if (T_ > 0) {
                tmem_load(tQ(m) + lanes + c, x);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0.f;
            }
            // A row that sees no key has no gradient, not even 0 times a key or lam that is not finite.
            if (none)
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0.f;
            if (live) store_row(dst + c, x, a.scale / f + nan, a.D - c, wide);
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        tmem_free(tmem, 512);
    }
    if (threadIdx.x == 0 && *gave_up) atomicOr(&g_gave_up_backward, 1u);
}

// ---- grad_k, grad_v, grad_table --------------------------------------------

template <int DP, int VP> struct GradKVShared {
    static constexpr int row = DP * 2;
    static constexpr int k = kOwn * row, v = kOwn * kBlock;       // one map, one block of 64 columns
    static constexpr int q = kStep * row, g = kStep * kBlock;
    static constexpr int stage = 2 * q + (VP / 64) * g;
    static constexpr int stages = 3;
    static constexpr int s = kOwn * kBlock;                       // P_0 - lam P_1 as an operand
    // Columns of tensor memory: two score tiles and e, grad_v, grad_k, s_m,
    // and with room for them (Dv of at most 64) v and the weights.
    static constexpr int c_s = 3 * kStep + VP + 2 * DP, c_v = c_s + kStep, c_w = c_v + VP / 2;
    static constexpr bool roomy = c_w + kStep / 2 <= 512;
    static_assert(c_v <= 512, "tensor memory");
    static constexpr int at_v = 2 * k, at_stage = at_v + (VP / 64) * v, at_w = at_stage + stages * stage,
                         bytes = at_w + (roomy ? 0 : s);
    static constexpr int table(int nb, int reach) { return nb ? 4 * (2 * reach + 1) + (2 * reach + 4) / 4 * 4 + 4 * 256 * nb : 0; }
};

// Per-query values of a step, the queries' positions among them.
struct alignas(16) QueryInfo {
    // Of each two queries: minus the log-sums of map 0, of map 1, minus d_0,
    // d_1, with the scales that the weights and s_m are formed with.
    float values[kStep / 2][8];
    int pos[kStep];
    int lo, hi;
};

struct KVBars {
    uint64_t kv_full, kv_ready, v_ready, fin, s_full, s_free, ds_full;
    uint64_t full[3], empty[3], ready[3];  // of a stage: loaded, free, cleared of idle queries
    uint32_t tmem, gave_up;
};

template <typename T, int DP, int VP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    dattn_grad_kv_tc_kernel(const __grid_constant__ DattnArgs a, const __grid_constant__ CUtensorMap mq,
                            const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                            const __grid_constant__ CUtensorMap mg)
{
    using F = GradKVShared<DP, VP>;
    constexpr int NS = F::stages;
    extern __shared__ unsigned char raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
    __shared__ KVBars bars;
    __shared__ QueryInfo infos[NS];
    const int span = 2 * a.reach + 1;
    // Bias of the head at hand by relative position, its bucket, and every
    // compute thread's own sums per bucket.
    float *table = reinterpret_cast<float *>(base + F::bytes);
    uint8_t *bucket = reinterpret_cast<uint8_t *>(table + span);
    float *sums = reinterpret_cast<float *>(bucket + (span + 3) / 4 * 4);

    const int warp = warp_number(), lane = threadIdx.x & 31;
    // The keys that most queries see first, of all heads and batch items.
    const int bn = blockIdx.x % (a.B * a.Hkv), b = bn / a.Hkv, n = bn - b * a.Hkv;
    const int key_tile = blockIdx.x / (a.B * a.Hkv), j0 = key_tile * kOwn;
    const int len = dattn_length(a, b);
    int first = 0;
    if (a.causal && !a.pos_q && !a.pos_k) first = min(max(j0 - (len - a.Lq), 0), a.Lq);
    const int per = j0 < len ? (a.Lq - first + kStep - 1) / kStep : 0;  // steps for each head
    const int T_ = per * a.G;

    if (threadIdx.x == 0) {
        bar_init(&bars.kv_full, 1);
        bar_init(&bars.kv_ready, 1);
        bar_init(&bars.v_ready, 8);
        bar_init(&bars.fin, 1);
        bar_init(&bars.s_full, 1);
        bar_init(&bars.s_free, 8);
        bar_init(&bars.ds_full, 8);
        for (int s = 0; s < NS; ++s) {
            bar_init(&bars.full[s], 1);
            bar_init(&bars.empty[s], 1);
            bar_init(&bars.ready[s], 1);
        }
        bars.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
        tma_prefetch(&mg);
    }
    if (warp == 9) tmem_alloc(&bars.tmem, 512);
    if (a.nb)
        for (int i = threadIdx.x; i < span; i += kBwdThreads)
            bucket[i] = static_cast<uint8_t>(min(max(a.bmap[i], 0), a.nb - 1));
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(bars.tmem);
    volatile uint32_t *gave_up = &bars.gave_up;
    auto tS = [&](int which) { return tmem + which * 64; };
    const uint32_t tV = tmem + 192;
    auto tK = [&](int m) { return tmem + 192 + VP + m * DP; };
    const uint32_t sbase = smem_addr(base);
    // Weights are formed times lift, s_m times lift * f.
    float lift = 1.f, f = 1.f;
    if (kScaled<T> && (warp < 8 || warp == 10)) {
        float most = 0.f;
        for (int g = lane; g < a.G; g += 32) most = fmaxf(most, fabsf(a.lam[n * a.G + g]));
#pragma unroll
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        lift = scale_to_range(1.f + most);
        f = scale_to_range(__uint_as_float(a.most[a.B * a.Hkv + bn]) * __uint_as_float(a.most[bn])) / lift;
    }

    if (warp == 8) {
        if (lane == 0 && T_ > 0) {
            bar_expect(&bars.kv_full, 2 * F::k + (VP / 64) * F::v);
            for (int m = 0; m < 2; ++m) tma_load(&mk, &bars.kv_full, base + m * F::k, 0, m, n, j0, b);
            for (int c = 0; c < VP / 64; ++c) tma_load(&mv, &bars.kv_full, base + F::at_v + c * F::v, c * 64, 0, n, j0, b);
            for (int t = 0; t < T_; ++t) {
                const int s = t % NS, h = n * a.G + t / per, l = first + (t % per) * kStep;
                unsigned char *st = base + F::at_stage + s * F::stage;
                bar_wait(&bars.empty[s], ((t / NS) & 1) ^ 1, gave_up);
                bar_expect(&bars.full[s], F::stage);
                for (int m = 0; m < 2; ++m) tma_load(&mq, &bars.full[s], st + m * F::q, 0, m, h, l, b);
                for (int c = 0; c < VP / 64; ++c) tma_load(&mg, &bars.full[s], st + 2 * F::q + c * F::g, c * 64, 0, h, l, b);
            }
            if (*gave_up) {
                bar_drain(&bars.kv_full, 0);
                for (int t = max(0, T_ - NS); t < T_; ++t) bar_drain(&bars.full[t % NS], (t / NS) & 1);
            }
        }
    } else if (warp == 9) {
        if (T_ > 0) {
            const bool issue = elect();
            constexpr uint32_t is = shape(is_bf16<T>, kStep, false), iv = shape(is_bf16<T>, VP, true),
                               ik = shape(is_bf16<T>, DP, true);
            const Operand<F::row> dk = along_row<F::row>(sbase), dq = along_row<F::row>(sbase + F::at_stage),
                                  dqr = over_rows<F::row>(sbase + F::at_stage, F::q);
            const Operand<128> dg = along_row<128>(sbase + F::at_stage + 2 * F::q),
                               dgr = over_rows<128>(sbase + F::at_stage + 2 * F::q, F::g), dw = along_row<128>(sbase + F::at_w), dv = along_row<128>(sbase + F::at_v);
            auto scores = [&](int t) {
                const uint32_t st = (t % NS) * F::stage;
                bar_wait_warp(&bars.ready[t % NS], (t / NS) & 1, gave_up);
                if (t > 0) bar_wait_warp(&bars.s_free, (t - 1) & 1, gave_up);
                fence_after();
                if (issue) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i)
                            mma_ss(tS(m), dk.at(m * F::k + i * 32), dq.at(st + m * F::q + i * 32), is, i > 0);
#pragma unroll
                    for (int i = 0; i < VP / 16; ++i) {
                        const uint64_t g = dg.at(st + (i / 4) * F::g + (i % 4) * 32);
                        if (F::roomy) mma_ts(tS(2), tmem + F::c_v + i * 8, g, is, i > 0);
                        else mma_ss(tS(2), dv.at((i / 4) * F::v + (i % 4) * 32), g, is, i > 0);
                    }
                    mma_commit(&bars.s_full);
                }
                __syncwarp();
            };
            bar_wait_warp(&bars.v_ready, 0, gave_up);
            scores(0);
            for (int t = 0; t < T_; ++t) {
                if (t + 1 < T_) scores(t + 1);
                bar_wait_warp(&bars.ds_full, t & 1, gave_up);
                fence_after();
                if (issue) {
                    const uint32_t st = (t % NS) * F::stage;
#pragma unroll
                    for (int i = 0; i < kStep / 16; ++i) {
                        const uint64_t g = dgr.at(st + i * 16 * 128);
                        if (F::roomy) mma_ts(tV, tmem + F::c_w + i * 8, g, iv, t > 0 || i > 0);
                        else mma_ss(tV, dw.at(i * 32), g, iv, t > 0 || i > 0);
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < kStep / 16; ++i)
                            mma_ts(tK(m), tmem + F::c_s + m * (kStep / 2) + i * 8, dqr.at(st + m * F::q + i * 16 * F::row), ik, t > 0 || i > 0);
                    mma_commit(&bars.empty[t % NS]);
                }
                __syncwarp();
            }
            if (issue) mma_commit(&bars.fin);
            bar_drain(&bars.fin, 0);
            __syncwarp();
        }
    } else if (warp == 10) {
        if (T_ > 0) {
            // Keys that are not to be used become zeros, once (past the
            // tensor's end TMA wrote them).
            bar_wait_warp(&bars.kv_full, 0, gave_up);
            bool any = false;
#pragma unroll
            for (int c = 0; c < kOwn / 32; ++c) {
                const int r = c * 32 + lane, j = j0 + r;
                if (j < a.Lk && (j >= len || (a.mask && !a.mask[static_cast<int64_t>(b) * a.Lk + j]))) {
                    clear_key<DP, VP>(base, r, F::k, F::at_v, F::v);
                    any = true;
                }
            }
            if (any) fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.kv_ready);
        }
        // A step ahead: the log-sums, d_m and positions of the lane's two queries.
        float next_lse[2][2], next_d[2][2];
        int next_pos[2];
        const auto fetch = [&](int t) {
            const int g = t / max(per, 1), h = n * a.G + g, l0 = first + (t - g * per) * kStep;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int l = l0 + c * 32 + lane;
                const bool in = t < T_ && l < a.Lq;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    next_lse[c][m] = in ? a.lse[((static_cast<int64_t>(b) * a.H + h) * 2 + m) * a.Lq + l] : INFINITY;
                    next_d[c][m] = in ? a.delta[((static_cast<int64_t>(b) * a.Hkv + n) * 2 + m) * a.rows + static_cast<int64_t>(l) * a.G + g] : 0.f;
                }
                next_pos[c] = !in ? 0 : a.pos_q ? a.pos_q[static_cast<int64_t>(b) * a.Lq + l] : len - a.Lq + l;
            }
        };
        fetch(0);
        const float higher = static_cast<float>(static_cast<int>(__float_as_uint(lift) >> 23) - 127);  // log2(lift)
        for (int t = 0; t < T_; ++t) {
            const int s = t % NS, l0 = first + (t % per) * kStep;
            QueryInfo &qi = infos[s];
            float lse[2][2], d[2][2];
            int pos[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    lse[c][m] = next_lse[c][m];
                    d[c][m] = next_d[c][m];
                }
                pos[c] = next_pos[c];
            }
            fetch(t + 1);
            bar_wait_warp(&bars.empty[s], ((t / NS) & 1) ^ 1, gave_up);
            int lo = INT32_MAX, hi = INT32_MIN;
            bool idle[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int i = c * 32 + lane;
                const bool in = l0 + i < a.Lq;
                // Pairs of queries: {map 0 of both, map 1 of both}.
                float *to = &qi.values[i >> 1][i & 1];
                to[0] = higher - lse[c][0];
                to[2] = higher - lse[c][1];
                to[4] = -d[c][0] * f;
                to[6] = -d[c][1] * f;
                qi.pos[i] = pos[c];
                idle[c] = in && lse[c][0] == INFINITY;
                if (in) {
                    lo = min(lo, pos[c]);
                    hi = max(hi, pos[c]);
                }
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            if (lane == 0) {
                qi.lo = lo;
                qi.hi = hi;
            }
            bar_wait_warp(&bars.full[s], (t / NS) & 1, gave_up);
            // Queries that see nothing take no part, whatever q and g hold.
            if (__any_sync(0xffffffffu, idle[0] || idle[1])) {
                unsigned char *st = base + F::at_stage + s * F::stage;
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (idle[c]) clear_key<DP, VP>(st, c * 32 + lane, F::q, 2 * F::q, F::g);
                fence_async();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.ready[s]);
        }
    } else {
        const int half = warp >> 2, rl = (warp & 3) * 32 + lane, tid = threadIdx.x;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int j = j0 + rl;
        const int64_t kat = static_cast<int64_t>(b) * a.Lk + j;
        const bool use = j < len && (!a.mask || a.mask[kat]);
        const int pos = use && a.pos_k ? a.pos_k[kat] : j;
        float *mine = sums + tid;
        if (T_ > 0) {
            bar_wait_warp(&bars.kv_full, 0, gave_up);
            bar_wait_warp(&bars.kv_ready, 0, gave_up);
            if (F::roomy) {
                for (int c = 0; c < VP / 64; ++c)
                    operand_to_tmem<128>(tmem + F::c_v + c * 32 + half * 16 + lanes, base + F::at_v + c * F::v, rl, half);
                tmem_store_wait();
                fence_before();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.v_ready);
        }
        for (int g = 0; g < a.G; ++g) {
            if (a.nb) {  // this head's bias, and sums from zero
                asm volatile("bar.sync 1, 256;" ::: "memory");
                for (int i = tid; i < span; i += 256) table[i] = a.table[bucket[i] * a.H + n * a.G + g] * kLog2e;
                for (int i = 0; i < a.nb; ++i) mine[i * 256] = 0.f;
                asm volatile("bar.sync 1, 256;" ::: "memory");
            }
            const float nlam = -a.lam[n * a.G + g];
            for (int u = 0; u < per; ++u) {
                const int t = g * per + u;
                const QueryInfo &qi = infos[t % NS];
                bar_wait_warp(&bars.s_full, t & 1, gave_up);
                fence_after();
                float e[32], x[2][32];
                tmem_load3(tS(2) + lanes + half * 32, tS(0) + lanes + half * 32, tS(1) + lanes + half * 32, e, x[0], x[1]);
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bars.s_free);
                const int rlo = pos - qi.hi, rhi = pos - qi.lo;
                const bool same = rlo >= a.reach || rhi <= -a.reach || rlo == rhi;  // one bucket for the whole step
                const bool even = !use || (!(a.causal && rhi > 0) && (a.nb == 0 || same));
                const bool fast = __all_sync(0xffffffffu, even);
                float add = 0.f, mul = a.scale_log2;
                int where = 0;
                if (a.nb) {
                    where = min(max(rlo, -a.reach), a.reach) + a.reach;
                    add = table[where];
                    where = bucket[where] * 256;
                }
                if (!use) add = -INFINITY;
                if (!fast) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int rel = pos - qi.pos[half * 32 + i];
                        const float bias = a.nb ? table[min(max(rel, -a.reach), a.reach) + a.reach] : 0.f;
                        const bool on = use && !(a.causal && rel > 0);
                        x[0][i] = on ? fmaf(x[0][i], mul, bias) : -INFINITY;
                        x[1][i] = on ? fmaf(x[1][i], mul, bias) : -INFINITY;
                    }
                    mul = 1.f;
                    add = 0.f;
                }
                const float2 mul_2 = {mul, mul}, add_2 = {add, add}, nl = {nlam, nlam}, f_2 = {f, f};
                const auto less_d = [&](float2 e, float2 nd) { return kScaled<T> ? fma2(e, f_2, nd) : add2(e, nd); };
                float2 total = {0.f, 0.f};
                uint32_t pw[16], p0[16], p1[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 lse = *reinterpret_cast<const float4 *>(&qi.values[half * 16 + i][0]);
                    const float4 nd = *reinterpret_cast<const float4 *>(&qi.values[half * 16 + i][4]);
                    const float2 l0 = {lse.x, lse.y}, l1 = {lse.z, lse.w}, d0 = {nd.x, nd.y}, d1 = {nd.z, nd.w};
                    const float2 ei = {e[2 * i], e[2 * i + 1]};
                    float2 w0 = fma2({x[0][2 * i], x[0][2 * i + 1]}, mul_2, add2(add_2, l0));
                    float2 w1 = fma2({x[1][2 * i], x[1][2 * i + 1]}, mul_2, add2(add_2, l1));
                    w0.x = ex2(w0.x);
                    w0.y = ex2(w0.y);
                    w1.x = ex2(w1.x);
                    w1.y = ex2(w1.y);
                    const float2 s0 = mul2(w0, less_d(ei, d0)), s1 = mul2(mul2(w1, nl), less_d(ei, d1)), w = fma2(w1, nl, w0);
                    const float2 both = add2(s0, s1);
                    total = add2(total, both);
                    x[0][2 * i] = both.x;  // kept for the buckets
                    x[0][2 * i + 1] = both.y;
                    pw[i] = pack2<T>(w.x, w.y);
                    p0[i] = pack2<T>(s0.x, s0.y);
                    p1[i] = pack2<T>(s1.x, s1.y);
                }
                if (a.nb && !fast) {
                    // Runs of one bucket are summed before they are added.
                    int last = bucket[min(max(pos - qi.pos[half * 32], -a.reach), a.reach) + a.reach];
                    float run = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int k = bucket[min(max(pos - qi.pos[half * 32 + i], -a.reach), a.reach) + a.reach];
                        if (k != last) {
                            mine[last * 256] += run;
                            run = 0.f;
                            last = k;
                        }
                        run += x[0][i];
                    }
                    mine[last * 256] += run;
                }
                if (t > 0) bar_wait_warp(&bars.empty[(t - 1) % NS], ((t - 1) / NS) & 1, gave_up);  // those of step t - 1 were used
                if (F::roomy) {
                    tmem_store(tmem + F::c_w + half * 16 + lanes, pw);
                } else {
                    store_operand(base + F::at_w, rl, half, pw);
                    fence_async();
                }
                tmem_store(tmem + F::c_s + half * 16 + lanes, p0);
                tmem_store(tmem + F::c_s + kStep / 2 + half * 16 + lanes, p1);
                tmem_store_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bars.ds_full);
                if (a.nb && fast) mine[where] += total.x + total.y;
            }
            if (a.nb) {
                asm volatile("bar.sync 1, 256;" ::: "memory");
                float *out = a.part_table + ((static_cast<int64_t>(b) * a.Hkv + n) * a.table_ctas + key_tile) * a.nb * a.G;
                for (int k = warp; k < a.nb; k += 8) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) s += sums[k * 256 + i * 32 + lane];
#pragma unroll
                    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                    if (lane == 0) out[k * a.G + g] = *gave_up ? NAN : s / (lift * f);
                }
            }
        }
        if (T_ > 0) bar_wait(&bars.fin, 0, gave_up);
        fence_after();
        const float nan = *gave_up ? NAN : 0.f;
        const bool in = j < a.Lk;
        const int64_t at = kat * a.Hkv + n;
        const bool wide_k = aligned16(a.grad_k), wide_v = aligned16(a.grad_v);
        // The warps of each half write half of grad_v's columns and one map of grad_k.
#pragma unroll 1
        for (int c = 0; c < VP / 2 + DP; c += 32) {
            const bool of_v = c < VP / 2;
            const int col = of_v ? half * (VP / 2) + c : c - VP / 2;
            float x[32];
            __syncwarp();
            if (T_ > 0) {
                tmem_load((of_v ? tV : tK(half)) + lanes + col, x);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0.f;
            }
            if (!in) continue;
            // A key that no query may see has no gradient, not even 0 times another's that is not finite.
            if (!use)
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0.f;
            if (of_v) store_row(static_cast<T *>(a.grad_v) + at * a.Dv + col, x, 1.f / lift + nan, a.Dv - col, wide_v);
            else store_row(static_cast<T *>(a.grad_k) + (at * 2 + half) * a.D + col, x, a.scale / (lift * f) + nan, a.D - col, wide_k);
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        tmem_free(tmem, 512);
    }
    if (threadIdx.x == 0 && *gave_up) atomicOr(&g_gave_up_backward, 1u);
}

struct BwdMaps {
    CUtensorMap q, k, v, g;
};

template <typename K>
cudaError_t launch_bwd(K kernel, dim3 grid, size_t smem, size_t most, const DattnArgs &a, const BwdMaps &m, cudaStream_t st)
{
    const cudaError_t e = allow_shared(kernel, most);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kBwdThreads, smem, st>>>(a, m.q, m.k, m.v, m.g);
    return cudaGetLastError();
}

template <typename T, int DP, int VP>
cudaError_t bwd_kernels(const DattnArgs &a, const BwdMaps &own_rows, const BwdMaps &own_keys, cudaStream_t st)
{
    using Q = GradQShared<DP, VP>;
    using KV = GradKVShared<DP, VP>;
    const int LP = kOwn / a.G;
    cudaError_t e = cudaSuccess;
    if (kScaled<T>) {
        const int heads = a.B * a.Hkv;
        e = cudaMemsetAsync(a.most, 0, sizeof(uint32_t) * 2 * heads, st);
        if (e != cudaSuccess) return e;
        dattn_most_v_kernel<<<static_cast<unsigned>((a.Lk + kMostKeys - 1) / kMostKeys) * heads, 256, 0, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    e = launch_bwd(dattn_grad_q_tc_kernel<T, DP, VP>, dim3((a.Lq + LP - 1) / LP * a.Hkv * a.B),
                   Q::bytes + 1024 + sizeof(float) * (a.nb ? a.G * (2 * a.reach + 1) : 0), Q::bytes + 1024 + sizeof(float) * kTcBiasBackward, a,
                   own_rows, st);
    if (e != cudaSuccess) return e;
    return launch_bwd(dattn_grad_kv_tc_kernel<T, DP, VP>, dim3((a.Lk + kOwn - 1) / kOwn * a.Hkv * a.B),
                      KV::bytes + 1024 + KV::table(a.nb, a.reach), KV::bytes + 1024 + KV::table(kTcBuckets, DATTN_MAX_REACH), a, own_keys, st);
}

template <typename T> cudaError_t bwd_widths(const DattnArgs &a, const BwdMaps &r, const BwdMaps &k, cudaStream_t st)
{
    if (a.D <= 32) return a.Dv <= 64 ? bwd_kernels<T, 32, 64>(a, r, k, st) : bwd_kernels<T, 32, 128>(a, r, k, st);
    return a.Dv <= 64 ? bwd_kernels<T, 64, 64>(a, r, k, st) : bwd_kernels<T, 64, 128>(a, r, k, st);
}

}  // namespace

uint32_t *dattn_gave_up_backward_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_gave_up_backward) == cudaSuccess ? static_cast<uint32_t *>(p) : nullptr;
}

da_status dattn_backward_tensor(const DattnArgs &a, int dtype, cudaStream_t st)
{
    const int wide = a.D <= 32 ? 32 : 64, LP = kOwn / a.G;
    const int64_t gl = static_cast<int64_t>(a.H) * a.Dv, gb = gl * a.Lq;  // strides of grad_out
    BwdMaps r, k;
    da_status e = DA_OK;
    auto make = [&](CUtensorMap &m, const void *p, int width, int maps, int heads, int len, const int64_t *s, int64_t s_map, int bw, int bh, int bl) {
        if (e == DA_OK) e = tensor_map(m, dtype, p, width, maps, heads, len, a.B, s_map, s[2], s[1], s[0], bw, bh, bl);
    };
    const int64_t gs[3] = {gb, gl, a.Dv};
    make(r.q, a.q, a.D, 2, a.H, a.Lq, a.qs, a.qs[3], wide, a.G, LP);
    make(r.g, a.grad_out, a.Dv, 1, a.H, a.Lq, gs, 0, 64, a.G, LP);
    make(r.k, a.k, a.D, 2, a.Hkv, a.Lk, a.ks, a.ks[3], wide, 1, kStep);
    make(r.v, a.v, a.Dv, 1, a.Hkv, a.Lk, a.vs, 0, 64, 1, kStep);
    make(k.q, a.q, a.D, 2, a.H, a.Lq, a.qs, a.qs[3], wide, 1, kStep);
    make(k.g, a.grad_out, a.Dv, 1, a.H, a.Lq, gs, 0, 64, 1, kStep);
    make(k.k, a.k, a.D, 2, a.Hkv, a.Lk, a.ks, a.ks[3], wide, 1, kOwn);
    make(k.v, a.v, a.Dv, 1, a.Hkv, a.Lk, a.vs, 0, 64, 1, kOwn);
    if (e != DA_OK) return e;
    const cudaError_t c = dtype == DA_BF16 ? bwd_widths<__nv_bfloat16>(a, r, k, st) : bwd_widths<__half>(a, r, k, st);
    return c == cudaSuccess ? DA_OK : cuda_fail(c, "differential attention backward launch");
}

}  // namespace da
