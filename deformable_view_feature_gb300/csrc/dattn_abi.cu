// extern "C" entry points of the differential attention (include/dattn.h):
// validation, the plan (kernels, split over the keys, workspace) and launches.
#include <cmath>

#include "dattn_tc.cuh"

namespace da {

da_status tensor_map(CUtensorMap &m, int dtype, const void *base, int width, int maps, int heads, int length, int batch,
                     int64_t s_map, int64_t s_head, int64_t s_len, int64_t s_batch, int box_width, int box_heads, int box_len)
{
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r{};
        return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
                       r == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<Encode>(f)
                   : nullptr;
    }();
    if (!encode) return fail(DA_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(maps), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(length), static_cast<cuuint64_t>(batch)};
    const int64_t s[4] = {s_map, s_head, s_len, s_batch};
    cuuint64_t strides[4];
    for (int i = 0; i < 4; ++i)  // the stride of a dimension of one is never used, but is checked
        strides[i] = dims[i + 1] == 1 ? 16 : static_cast<cuuint64_t>(s[i]) * 2;
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(box_width), 1, static_cast<cuuint32_t>(box_heads),
                               static_cast<cuuint32_t>(box_len), 1};
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    const CUresult r = encode(&m, dtype == DA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                              const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              box_width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? DA_OK : fail(DA_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", static_cast<int>(r));
}

namespace {

// The tensor-core kernels' rule. 16-bit types; widths that their tiles hold
// and whose rows are multiples of 16 bytes; the group of heads within a tile
// and its expanded bias within 32 KB; and what a TMA box needs: 16-byte
// aligned addresses and strides, none of them zero.
// The backward kernels' shared memory leaves room for half of that bias, and
// for sums of at most 32 buckets.
bool tensor_serves(const dattn_problem &d, bool backward)
{
    if (d.dtype != DA_BF16 && d.dtype != DA_F16) return false;
    const int G = d.num_heads / d.num_kv_heads;
    if (d.width % 8 || d.value_width % 8 || d.width > 64 || d.value_width > 128 || G > 128) return false;
    if (d.batch < 1 || d.num_queries < 1 || d.num_keys < 1) return false;
    if (G * (2 * (d.num_buckets > 0 ? d.reach : 0) + 129) > (backward ? 4096 : 8192)) return false;
    // Their grids are one-dimensional.
    const int64_t tiles = (static_cast<int64_t>(d.num_queries > d.num_keys ? d.num_queries : d.num_keys) * G / 64 + 1);
    if (tiles * d.batch * d.num_kv_heads > INT32_MAX / 4) return false;
    if (backward && d.num_buckets > 32) return false;
    if (!aligned(d.q, 16) || !aligned(d.k, 16) || !aligned(d.v, 16)) return false;
    const int nq[4] = {d.batch, d.num_queries, d.num_heads, 2}, nk[4] = {d.batch, d.num_keys, d.num_kv_heads, 2};
    auto fits = [](int64_t stride, int size) { return size == 1 || (stride > 0 && stride % 8 == 0 && stride < (int64_t{1} << 38)); };
    for (int i = 0; i < 4; ++i)
        if (!fits(d.q_stride[i], nq[i]) || !fits(d.k_stride[i], nk[i]) || (i < 3 && !fits(d.v_stride[i], nk[i]))) return false;
    return true;
}

struct DattnPlan {
    DattnArgs a;
    int elem;
    bool tensor;
    size_t part_o, part_ml, part_kv, delta, part_table, most, total;
};

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// CTAs to share a tile where the tiles alone leave SMs without work: enough
// that each of the 152 SMs has its `resident` ones, each with at least one
// of the `steps` that a tile's walk has.
int split_count(int64_t tiles, int64_t steps, int resident)
{
    const int64_t want = tiles > 0 ? 152 * resident / tiles : 1;
    const int64_t n = want < steps ? want : steps;
    return static_cast<int>(n < 1 ? 1 : n);
}

da_status dattn_plan(const dattn_problem *pr, bool backward, DattnPlan &p)
{
    if (!pr) return fail(DA_ERR_NULL, "problem is NULL");
    const dattn_problem &d = *pr;
    if (d.batch < 0 || d.num_queries < 0 || d.num_keys < 0) return fail(DA_ERR_SHAPE, "negative size");
    if (d.num_heads < 1 || d.num_kv_heads < 1 || d.num_heads % d.num_kv_heads != 0)
        return fail(DA_ERR_SHAPE, "num_heads (%d) must be a positive multiple of num_kv_heads (%d)", d.num_heads,
                    d.num_kv_heads);
    if (d.width < 1 || d.value_width < 1) return fail(DA_ERR_SHAPE, "width %d and value_width %d must be positive", d.width, d.value_width);
    if (d.width > DATTN_MAX_WIDTH || d.value_width > DATTN_MAX_VALUE_WIDTH)
        return fail(DA_ERR_UNSUPPORTED, "width %d or value_width %d exceeds %d or %d", d.width, d.value_width,
                    DATTN_MAX_WIDTH, DATTN_MAX_VALUE_WIDTH);
    if (d.dtype != DA_F32 && d.dtype != DA_BF16 && d.dtype != DA_F16) return fail(DA_ERR_SHAPE, "unknown dtype %d", d.dtype);
    if (!std::isfinite(d.scale)) return fail(DA_ERR_SHAPE, "scale must be finite");
    if (d.batch > 65535 || d.num_kv_heads > 65535) return fail(DA_ERR_UNSUPPORTED, "batch or num_kv_heads exceeds 65535");
    const int G = d.num_heads / d.num_kv_heads;
    const int64_t rows = static_cast<int64_t>(d.num_queries) * G;
    if (rows > INT32_MAX - 1024 || d.num_keys > INT32_MAX - 1024 || d.num_queries > (1 << 29) || d.num_keys > (1 << 29))
        return fail(DA_ERR_UNSUPPORTED, "sequences too long: %d queries, %d keys", d.num_queries, d.num_keys);
    if (d.num_buckets < 0) return fail(DA_ERR_SHAPE, "negative num_buckets");
    if (d.num_buckets > 0) {
        if (d.reach < 1) return fail(DA_ERR_SHAPE, "reach %d must be positive", d.reach);
        if (d.reach > DATTN_MAX_REACH) return fail(DA_ERR_UNSUPPORTED, "reach %d exceeds %d", d.reach, DATTN_MAX_REACH);
        if (static_cast<int64_t>(d.num_buckets) * G > DATTN_MAX_TABLE)
            return fail(DA_ERR_UNSUPPORTED, "num_buckets * num_heads / num_kv_heads = %lld exceeds %d",
                        static_cast<long long>(d.num_buckets) * G, DATTN_MAX_TABLE);
    }
    for (int i = 0; i < 4; ++i)
        if (d.q_stride[i] < 0 || d.k_stride[i] < 0 || (i < 3 && d.v_stride[i] < 0))
            return fail(DA_ERR_SHAPE, "strides must not be negative");
    DattnArgs &a = p.a;
    a.q = d.q;
    a.k = d.k;
    a.v = d.v;
    for (int i = 0; i < 4; ++i) {
        a.qs[i] = d.q_stride[i];
        a.ks[i] = d.k_stride[i];
        if (i < 3) a.vs[i] = d.v_stride[i];
    }
    a.lam = d.lam;
    a.table = d.bias_table;
    a.bmap = d.bucket_map;
    a.pos_q = d.pos_q;
    a.pos_k = d.pos_k;
    a.lengths = d.key_lengths;
    a.mask = d.key_mask;
    a.B = d.batch;
    a.Lq = d.num_queries;
    a.Lk = d.num_keys;
    a.H = d.num_heads;
    a.Hkv = d.num_kv_heads;
    a.G = G;
    a.D = d.width;
    a.Dv = d.value_width;
    a.nb = d.num_buckets;
    a.reach = d.num_buckets > 0 ? d.reach : 0;
    a.causal = d.causal != 0;
    a.rows = static_cast<int32_t>(rows);
    a.div_G = FastDiv::make(static_cast<uint32_t>(G));
    a.scale = d.scale;
    a.scale_log2 = static_cast<float>(static_cast<double>(d.scale) * 1.4426950408889634);
    a.wide = d.dtype == DA_F32 && d.width % 4 == 0 && d.value_width % 4 == 0 && aligned(d.q, 16) && aligned(d.k, 16) && aligned(d.v, 16);
    for (int i = 0; i < 4; ++i) a.wide = a.wide && a.qs[i] % 4 == 0 && a.ks[i] % 4 == 0 && (i == 3 || a.vs[i] % 4 == 0);
    p.elem = d.dtype == DA_F32 ? 4 : 2;
    p.tensor = tensor_serves(d, backward);
    const int64_t bn = static_cast<int64_t>(a.B) * a.Hkv;
    size_t at = 0;
    a.splits = a.row_splits = 1;
    a.keys_per_split = a.Lk > 0 ? a.Lk : 1;
    const auto split_keys = [&](int64_t tiles, int least, int resident) {
        const int n = split_count(tiles, a.Lk / least, resident);
        if (n > 1) {
            a.keys_per_split = ((a.Lk + n - 1) / n + 63) / 64 * 64;
            a.splits = (a.Lk + a.keys_per_split - 1) / a.keys_per_split;
        }
    };
    if (!backward) {
        // A tensor-core CTA fills an SM, two of the general ones fit.
        const int qt = p.tensor ? 128 / G * G : dattn_general_row_tile(a);
        split_keys(bn * ((rows + qt - 1) / qt), 128, p.tensor ? 1 : 2);
        if (a.splits > 1) {
            p.part_o = at;
            at += round256(sizeof(float) * bn * rows * a.splits * 2 * a.Dv);
            p.part_ml = at;
            at += round256(sizeof(float) * bn * rows * a.splits * 4);
        }
    } else {
        // Sized for the general kernels, which also take over where grad_out
        // turns out not to be aligned.
        const int tile = dattn_general_tile(a);
        const int64_t key_tiles = (a.Lk + tile - 1) / tile, row_tiles = (rows + tile - 1) / tile;
        split_keys(bn * row_tiles, tile, 2);
        a.row_splits = split_count(bn * key_tiles, row_tiles, 1);  // one CTA fills an SM's shared memory
        a.table_ctas = static_cast<int32_t>(key_tiles * a.row_splits);
        if (a.splits > 1) {
            p.part_o = at;
            at += round256(sizeof(float) * bn * rows * a.splits * 2 * a.D);
            p.part_ml = at;
            at += round256(sizeof(float) * bn * rows * a.splits * 2);
        }
        if (a.row_splits > 1) {
            p.part_kv = at;
            at += round256(sizeof(float) * bn * a.Lk * a.row_splits * (a.Dv + 2 * a.D));
        }
        p.delta = at;
        at += round256(sizeof(float) * bn * 2 * rows);
        p.part_table = at;
        at += round256(sizeof(float) * bn * a.table_ctas * a.nb * G);
        p.most = at;
        if (p.tensor && d.dtype == DA_F16) at += round256(sizeof(uint32_t) * 2 * bn);
    }
    p.total = at;
    return DA_OK;
}

da_status dattn_buffers(DattnPlan &p, void *ws, size_t ws_bytes)
{
    DattnArgs &a = p.a;
    const int64_t nq = static_cast<int64_t>(a.B) * a.rows, nk = static_cast<int64_t>(a.B) * a.Lk;
    if ((nq > 0 && !a.q) || (nk > 0 && (!a.k || !a.v))) return fail(DA_ERR_NULL, "q, k or v is NULL");
    if (!a.lam) return fail(DA_ERR_NULL, "lam is NULL");
    if (a.nb > 0 && (!a.table || !a.bmap)) return fail(DA_ERR_NULL, "bias_table or bucket_map is NULL");
    const void *elems[] = {a.q, a.k, a.v, a.out, a.out1, a.grad_out, a.grad_q, a.grad_k, a.grad_v};
    for (const void *x : elems)
        if (!aligned(x, p.elem)) return fail(DA_ERR_ALIGN, "q, k, v, outputs and gradients must be aligned to their elements");
    const void *words[] = {a.lam, a.table, a.bmap, a.pos_q, a.pos_k, a.lengths, a.lse, a.grad_lam, a.grad_table};
    for (const void *x : words)
        if (!aligned(x, 4)) return fail(DA_ERR_ALIGN, "fp32 and int32 tensors must be 4-byte aligned");
    if (p.total > 0) {
        if (!ws || ws_bytes < p.total)
            return fail(DA_ERR_WORKSPACE, "workspace of %zu bytes; %zu are needed", ws ? ws_bytes : size_t{0}, p.total);
        if (!aligned(ws, 256)) return fail(DA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    }
    char *w = static_cast<char *>(ws);
    a.part_o = reinterpret_cast<float *>(w + p.part_o);
    a.part_ml = reinterpret_cast<float *>(w + p.part_ml);
    a.part_kv = reinterpret_cast<float *>(w + p.part_kv);
    a.delta = reinterpret_cast<float *>(w + p.delta);
    a.part_table = reinterpret_cast<float *>(w + p.part_table);
    a.most = reinterpret_cast<uint32_t *>(w + p.most);
    return DA_OK;
}

}  // namespace
}  // namespace da

extern "C" {

int32_t dattn_path(const dattn_problem *p, int32_t backward)
{
    da::DattnPlan pl{};
    return da::dattn_plan(p, backward != 0, pl) == DA_OK ? static_cast<int32_t>(pl.tensor) : -1;
}

da_status dattn_workspace_size(const dattn_problem *p, int32_t backward, size_t *bytes)
{
    if (!bytes) return da::fail(DA_ERR_NULL, "bytes is NULL");
    da::DattnPlan pl{};
    const da_status st = da::dattn_plan(p, backward != 0, pl);
    if (st == DA_OK) *bytes = pl.total;
    return st;
}

da_status dattn_forward(const dattn_problem *p, void *out, void *out1, float *lse, void *workspace,
                        size_t workspace_bytes, da_stream_t stream)
{
    da::DattnPlan pl{};
    da_status st = da::dattn_plan(p, false, pl);
    if (st != DA_OK) return st;
    pl.a.out = out;
    pl.a.out1 = out1;
    pl.a.lse = lse;
    if ((st = da::dattn_buffers(pl, workspace, workspace_bytes)) != DA_OK) return st;
    if (static_cast<int64_t>(pl.a.B) * pl.a.rows == 0) return DA_OK;
    if (!out) return da::fail(DA_ERR_NULL, "out is NULL");
    if ((out1 == nullptr) != (lse == nullptr)) return da::fail(DA_ERR_NULL, "out1 and lse go together");
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (pl.tensor) {
        if ((st = da::dattn_forward_tensor(pl.a, p->dtype, cs)) != DA_OK) return st;
    }
    cudaError_t e = pl.tensor ? cudaSuccess : da::dattn_forward_general(pl.a, p->dtype, cs);
    if (e == cudaSuccess && pl.a.splits > 1) e = da::dattn_merge(pl.a, p->dtype, cs);
    return e == cudaSuccess ? DA_OK : da::cuda_fail(e, "differential attention launch");
}

da_status dattn_backward(const dattn_problem *p, const void *out, const void *out1, const float *lse,
                         const void *grad_out, void *grad_q, void *grad_k, void *grad_v, float *grad_lam,
                         float *grad_table, void *workspace, size_t workspace_bytes, da_stream_t stream)
{
    da::DattnPlan pl{};
    da_status st = da::dattn_plan(p, true, pl);
    if (st != DA_OK) return st;
    da::DattnArgs &a = pl.a;
    a.out = const_cast<void *>(out);
    a.out1 = const_cast<void *>(out1);
    a.lse = const_cast<float *>(lse);
    a.grad_out = grad_out;
    a.grad_q = grad_q;
    a.grad_k = grad_k;
    a.grad_v = grad_v;
    a.grad_lam = grad_lam;
    a.grad_table = grad_table;
    if ((st = da::dattn_buffers(pl, workspace, workspace_bytes)) != DA_OK) return st;
    if (static_cast<int64_t>(a.B) * a.rows > 0 && (!out || !out1 || !lse || !grad_out || !grad_q))
        return da::fail(DA_ERR_NULL, "out, out1, lse, grad_out or grad_q is NULL");
    if (static_cast<int64_t>(a.B) * a.Lk > 0 && (!grad_k || !grad_v)) return da::fail(DA_ERR_NULL, "grad_k or grad_v is NULL");
    if (!grad_lam || (a.nb > 0 && !grad_table)) return da::fail(DA_ERR_NULL, "grad_lam or grad_table is NULL");
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    a.wide = a.wide && da::aligned(grad_out, 16);
    if (pl.tensor && da::aligned(grad_out, 16) && da::aligned(out, 16) && da::aligned(out1, 16)) {
        a.table_ctas = (a.Lk + 127) / 128;
        if ((st = da::dattn_backward_tensor(a, p->dtype, cs)) != DA_OK) return st;
    } else if (a.B > 0) {
        e = da::dattn_backward_general(a, p->dtype, cs);
    }
    if (e == cudaSuccess) e = da::dattn_finish_backward(a, cs);
    return e == cudaSuccess ? DA_OK : da::cuda_fail(e, "differential attention backward launch");
}

da_status dattn_device_status(uint32_t *gave_up, da_stream_t stream)
{
    if (!gave_up) return da::fail(DA_ERR_NULL, "gave_up is NULL");
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    uint32_t *words[2] = {da::dattn_gave_up_word(), da::dattn_gave_up_backward_word()}, got[2] = {0, 0};
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
        if (!words[i]) return da::cuda_fail(cudaGetLastError(), "address of a status word");
        e = cudaMemcpyAsync(&got[i], words[i], sizeof got[i], cudaMemcpyDeviceToHost, cs);
        if (e == cudaSuccess) e = cudaMemsetAsync(words[i], 0, sizeof got[i], cs);
    }
    if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
    *gave_up = got[0] | got[1];
    return e == cudaSuccess ? DA_OK : da::cuda_fail(e, "status word");
}

}  // extern "C"
