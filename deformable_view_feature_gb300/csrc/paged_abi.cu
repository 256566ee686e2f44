// extern "C" entry points of the paged cache (include/paged.h): validation,
// the plan (kernels, workspace) and launches.
#include <cmath>

#include "paged_internal.cuh"
#include "qkr_internal.cuh"

namespace da {
namespace {

da_status check_cache(const pg_cache &c, int batch, int elem)
{
    if (c.num_pages < 0 || c.table_pages < 0) return fail(DA_ERR_SHAPE, "negative size of the cache");
    if (c.page_size < 1) return fail(DA_ERR_SHAPE, "page_size %d must be positive", c.page_size);
    if (static_cast<int64_t>(c.table_pages) * c.page_size >= (1 << 29))
        return fail(DA_ERR_UNSUPPORTED, "sequences of 2^29 places or more");
    for (int i = 0; i < 4; ++i)
        if (c.k_stride[i] < 0 || (i < 3 && c.v_stride[i] < 0)) return fail(DA_ERR_SHAPE, "strides must not be negative");
    if (!aligned(c.k, elem) || !aligned(c.v, elem)) return fail(DA_ERR_ALIGN, "the cache must be aligned to its elements");
    if (!aligned(c.page_table, 4) || !aligned(c.lengths, 4) || !aligned(c.counts, 4))
        return fail(DA_ERR_ALIGN, "int32 tensors must be 4-byte aligned");
    if (batch > 0 && !c.lengths) return fail(DA_ERR_NULL, "lengths is NULL");
    if (batch > 0 && c.table_pages > 0 && !c.page_table) return fail(DA_ERR_NULL, "page_table is NULL");
    return DA_OK;
}

// The tensor-core kernel's rule. 16-bit types; widths that its tiles hold and
// whose rows are multiples of 16 bytes; a group of heads within a tile; pages of
// whole groups of eight places, by which shared memory is swizzled; a bias (of all
// heads) that it has room for; and what a TMA box needs: 16-byte aligned addresses
// and strides, none of them zero. Over four caches of up to 8,192 keys (2 key heads,
// D = 64, bf16) it takes 25 us for 4 rows, 31 for 64 and 79 for 1,024 in a replayed
// graph; outside the rule, with pages of 20, the fp32 units take 36, 165 and 1,803.
bool tensor_serves(const pg_problem &d)
{
    const pg_cache &c = d.cache;
    if (d.dtype != DA_BF16 && d.dtype != DA_F16) return false;
    if (d.width % 8 || d.value_width % 8 || d.width > 64 || d.value_width > 128 || d.num_heads / d.num_kv_heads > 64) return false;
    if (c.page_size % 8 || c.num_pages < 1 || c.table_pages < 1 || d.batch < 1 || d.num_tokens < 1) return false;
    if (d.num_buckets > 0 && paged_bias_bytes(d.num_buckets, d.num_heads, d.reach) > kPgBias) return false;
    if (!aligned(d.q, 16) || !aligned(c.k, 16) || !aligned(c.v, 16)) return false;
    const int nq[4] = {d.batch, d.num_tokens, d.num_heads, 2}, nk[4] = {c.num_pages, c.page_size, d.num_kv_heads, 2};
    auto fits = [](int64_t stride, int size) { return size == 1 || (stride > 0 && stride % 8 == 0 && stride < (int64_t{1} << 38)); };
    for (int i = 0; i < 4; ++i)
        if (!fits(d.q_stride[i], nq[i]) || !fits(c.k_stride[i], nk[i]) || (i < 3 && !fits(c.v_stride[i], nk[i]))) return false;
    return true;
}

// Up to here rows are taken straight from memory. Four caches of 8,192 keys in
// fp32 (2 key heads, D = 64) take 26, 55, 79 and 95 us so for 4, 8, 12 and 16
// rows, and 73 us each in tiles.
constexpr int kFewRows = 8;

struct PagedPlan {
    DattnArgs a;
    PagedTcArgs tc;
    size_t part_o, part_ml, slots, total;
    bool tensor, few, quads;
};

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

da_status paged_plan(const pg_problem *pr, PagedPlan &p)
{
    if (!pr) return fail(DA_ERR_NULL, "problem is NULL");
    const pg_problem &d = *pr;
    const pg_cache &c = d.cache;
    if (d.batch < 0 || d.num_tokens < 0) return fail(DA_ERR_SHAPE, "negative size");
    if (d.num_heads < 1 || d.num_kv_heads < 1 || d.num_heads % d.num_kv_heads != 0)
        return fail(DA_ERR_SHAPE, "num_heads (%d) must be a positive multiple of num_kv_heads (%d)", d.num_heads, d.num_kv_heads);
    if (d.width < 1 || d.value_width < 1) return fail(DA_ERR_SHAPE, "width %d and value_width %d must be positive", d.width, d.value_width);
    if (d.width > DATTN_MAX_WIDTH || d.value_width > DATTN_MAX_VALUE_WIDTH)
        return fail(DA_ERR_UNSUPPORTED, "width %d or value_width %d exceeds %d or %d", d.width, d.value_width, DATTN_MAX_WIDTH,
                    DATTN_MAX_VALUE_WIDTH);
    if (d.dtype != DA_F32 && d.dtype != DA_BF16 && d.dtype != DA_F16) return fail(DA_ERR_SHAPE, "unknown dtype %d", d.dtype);
    if (!std::isfinite(d.scale)) return fail(DA_ERR_SHAPE, "scale must be finite");
    if (d.batch > 65535 || d.num_kv_heads > 65535) return fail(DA_ERR_UNSUPPORTED, "batch or num_kv_heads exceeds 65535");
    const int G = d.num_heads / d.num_kv_heads, elem = d.dtype == DA_F32 ? 4 : 2;
    const int64_t rows = static_cast<int64_t>(d.num_tokens) * G;
    if (rows > (1 << 29) || static_cast<int64_t>(d.batch) * d.num_kv_heads * rows > INT32_MAX)
        return fail(DA_ERR_UNSUPPORTED, "too many rows: %d tokens of %d heads in %d sequences", d.num_tokens, d.num_heads, d.batch);
    if (d.num_buckets < 0) return fail(DA_ERR_SHAPE, "negative num_buckets");
    if (d.num_buckets > 0) {
        if (d.reach < 1) return fail(DA_ERR_SHAPE, "reach %d must be positive", d.reach);
        if (d.reach > DATTN_MAX_REACH) return fail(DA_ERR_UNSUPPORTED, "reach %d exceeds %d", d.reach, DATTN_MAX_REACH);
        if (static_cast<int64_t>(d.num_buckets) * G > DATTN_MAX_TABLE)
            return fail(DA_ERR_UNSUPPORTED, "num_buckets * num_heads / num_kv_heads = %lld exceeds %d",
                        static_cast<long long>(d.num_buckets) * G, DATTN_MAX_TABLE);
    }
    for (int i = 0; i < 4; ++i)
        if (d.q_stride[i] < 0) return fail(DA_ERR_SHAPE, "strides must not be negative");
    const da_status st = check_cache(c, d.batch, elem);
    if (st != DA_OK) return st;
    DattnArgs &a = p.a;
    a = DattnArgs{};
    a.pg = {c.page_table, c.counts, d.tree, c.table_pages, c.page_size, c.num_pages, FastDiv::make(static_cast<uint32_t>(c.page_size))};
    a.q = d.q;
    a.k = c.k;
    a.v = c.v;
    for (int i = 0; i < 4; ++i) {
        a.qs[i] = d.q_stride[i];
        a.ks[i] = c.k_stride[i];
        if (i < 3) a.vs[i] = c.v_stride[i];
    }
    a.lam = d.lam;
    a.table = d.bias_table;
    a.bmap = d.bucket_map;
    a.pos_q = d.pos_q;
    a.pos_k = d.pos_k;
    a.lengths = c.lengths;
    a.mask = d.key_mask;
    a.B = d.batch;
    a.Lq = d.num_tokens;
    a.Lk = c.table_pages * c.page_size;
    a.H = d.num_heads;
    a.Hkv = d.num_kv_heads;
    a.G = G;
    a.D = d.width;
    a.Dv = d.value_width;
    a.nb = d.num_buckets;
    a.reach = d.num_buckets > 0 ? d.reach : 0;
    a.causal = d.causal != 0 && !d.tree;
    a.rows = static_cast<int32_t>(rows);
    a.div_G = FastDiv::make(static_cast<uint32_t>(G));
    a.scale = d.scale;
    a.scale_log2 = static_cast<float>(static_cast<double>(d.scale) * 1.4426950408889634);
    a.wide = d.dtype == DA_F32 && d.width % 4 == 0 && d.value_width % 4 == 0 && aligned(d.q, 16) && aligned(c.k, 16) && aligned(c.v, 16);
    for (int i = 0; i < 4; ++i) a.wide = a.wide && a.qs[i] % 4 == 0 && a.ks[i] % 4 == 0 && (i == 3 || a.vs[i] % 4 == 0);
    p.part_o = p.part_ml = p.slots = p.total = 0;
    a.splits = 1;
    a.keys_per_split = a.Lk > 0 ? a.Lk : 1;
    p.tensor = tensor_serves(d);
    if (p.tensor) {
        // Rows of a tile. Four caches of 8,192 keys (2 key heads, D = 64, bf16) take
        // 24 us with 16 or 32 for 16 rows and 28 with 64; 27.0 with 16, 26.9 with 32
        // and 29.0 with 64 for 32 rows; 33, 29.8 and 29.5 for 64, where 32 is taken
        // because its weights carry what their rounding took. 124 rows take 40 us
        // with 32 and 35 with 64, 4,084 rows 298 and 124.
        PagedTcArgs &t = p.tc;
        t.RT = rows <= 16 ? 16 : rows <= 64 && G <= 32 ? 32 : 64;
        t.LP = t.RT / G;
        t.row_tiles = (d.num_tokens + t.LP - 1) / t.LP;
        t.box = 8;
        while (t.box < 128 && c.page_size % (2 * t.box) == 0) t.box *= 2;
        const int64_t tiles = static_cast<int64_t>(d.batch) * d.num_kv_heads * t.row_tiles, steps = tiles * ((a.Lk + 127) / 128);
        if (steps / 152 >= INT32_MAX / 2) return fail(DA_ERR_UNSUPPORTED, "too many rows and keys");
        t.ctas = static_cast<int32_t>(steps < 152 ? steps : 152);  // one fills an SM
        p.total += round256(sizeof(float) * 2 * t.ctas * t.RT * 2 * a.Dv);
        p.part_ml = p.total;
        p.total += round256(sizeof(float) * 2 * t.ctas * t.RT * 4);
        p.slots = p.total;
        p.total += round256(sizeof(int32_t) * 4 * t.ctas);
        return DA_OK;
    }
    // CTAs to share a tile where tiles alone leave SMs without work: two to an SM
    // with 64 keys or more of a full table each (73 us for 16 rows over 8,192 keys
    // four times in fp32, four to an SM 83); of the few rows' CTAs twice as many, so
    // that sequences' different lengths leave fewer SMs idle, with 256 keys or
    // more, 32 for each warp (26 us for 4 rows; with 64 keys or more 40).
    p.few = rows <= kFewRows;
    p.quads = d.width % 4 == 0 && d.value_width % 4 == 0 && aligned(d.q, 4 * elem) && aligned(c.k, 4 * elem) && aligned(c.v, 4 * elem);
    for (int i = 0; i < 4; ++i) p.quads = p.quads && a.qs[i] % 4 == 0 && a.ks[i] % 4 == 0 && (i == 3 || a.vs[i] % 4 == 0);
    const int64_t bn = static_cast<int64_t>(a.B) * a.Hkv, qt = p.few ? rows : dattn_general_row_tile(a), tiles = rows > 0 ? bn * ((rows + qt - 1) / qt) : 0;
    if (tiles > 0) {
        const int64_t want = 152 * (p.few ? 4 : 2) / tiles, steps = a.Lk / (p.few ? 256 : 64), n = want < steps ? want : steps;
        a.splits = static_cast<int32_t>(n < 1 ? 1 : n);
    }
    if (a.splits > 1) {
        p.part_o = p.total;
        p.total += round256(sizeof(float) * bn * rows * a.splits * 2 * a.Dv);
        p.part_ml = p.total;
        p.total += round256(sizeof(float) * bn * rows * a.splits * 4);
    }
    return DA_OK;
}

}  // namespace
}  // namespace da

extern "C" {

da_status pg_append(const qkr_problem *p, const void *v, const int64_t *v_stride, int32_t value_width, const pg_cache *cache,
                    void *out_q, da_stream_t stream)
{
    if (!p || !v_stride || !cache) return da::fail(DA_ERR_NULL, "problem, v_stride or cache is NULL");
    da::QkrArgs a{};
    da_status st = da::qkr_sides(p, out_q, nullptr, a);
    if (st != DA_OK) return st;
    const int elem = p->dtype == DA_F32 ? 4 : 2, T = p->num_keys;
    if (p->num_queries != 0 && p->num_queries != T)
        return da::fail(DA_ERR_SHAPE, "num_queries (%d) must be 0 or num_keys (%d)", p->num_queries, T);
    if (value_width < 1) return da::fail(DA_ERR_SHAPE, "value_width %d must be positive", value_width);
    if (value_width > DATTN_MAX_VALUE_WIDTH) return da::fail(DA_ERR_UNSUPPORTED, "value_width %d exceeds %d", value_width, DATTN_MAX_VALUE_WIDTH);
    for (int i = 0; i < 3; ++i)
        if (v_stride[i] < 0) return da::fail(DA_ERR_SHAPE, "strides must not be negative");
    if ((st = da::check_cache(*cache, p->batch, elem)) != DA_OK) return st;
    if (!da::aligned(v, elem)) return da::fail(DA_ERR_ALIGN, "v must be aligned to its elements");
    if (a.sides == 0) return DA_OK;
    const bool places = cache->num_pages > 0 && cache->table_pages > 0;
    if (!v || (places && (!cache->k || !cache->v))) return da::fail(DA_ERR_NULL, "v or the cache is NULL");
    if (p->num_queries > 0 && !out_q) return da::fail(DA_ERR_NULL, "out_q is NULL");
    da::QkrSide &k = a.side[a.sides - 1], &s = a.side[a.sides];
    k.y = cache->k;
    s = k;
    k.paged = s.paged = 1;
    for (int i = 0; i < 4; ++i) k.ys[i] = cache->k_stride[i];
    s.x = v;
    s.y = cache->v;
    s.M = 1;
    s.D = value_width;
    s.R = s.normed = 0;
    s.w = nullptr;
    for (int i = 0; i < 3; ++i) {
        s.xs[i] = v_stride[i];
        s.ys[i] = cache->v_stride[i];
    }
    s.xs[3] = s.ys[3] = 0;
    ++a.sides;
    a.table = cache->page_table;
    a.lengths = cache->lengths;
    a.counts = cache->counts;
    a.table_pages = cache->table_pages;
    a.page_size = cache->page_size;
    a.num_pages = cache->num_pages;
    a.div_page = da::FastDiv::make(static_cast<uint32_t>(cache->page_size));
    return da::qkr_launch_forward(a, p->dtype, reinterpret_cast<cudaStream_t>(stream));
}

int32_t pg_path(const pg_problem *p)
{
    da::PagedPlan pl{};
    return da::paged_plan(p, pl) == DA_OK ? static_cast<int32_t>(pl.tensor) : -1;
}

da_status pg_workspace_size(const pg_problem *p, size_t *bytes)
{
    if (!bytes) return da::fail(DA_ERR_NULL, "bytes is NULL");
    da::PagedPlan pl{};
    const da_status st = da::paged_plan(p, pl);
    if (st == DA_OK) *bytes = pl.total;
    return st;
}

da_status pg_attention(const pg_problem *p, void *out, void *workspace, size_t workspace_bytes, da_stream_t stream)
{
    da::PagedPlan pl{};
    da_status st = da::paged_plan(p, pl);
    if (st != DA_OK) return st;
    da::DattnArgs &a = pl.a;
    const int elem = p->dtype == DA_F32 ? 4 : 2;
    if (!da::aligned(a.q, elem) || !da::aligned(out, elem)) return da::fail(DA_ERR_ALIGN, "q and out must be aligned to their elements");
    const void *words[] = {a.lam, a.table, a.bmap, a.pos_q, a.pos_k};
    for (const void *x : words)
        if (!da::aligned(x, 4)) return da::fail(DA_ERR_ALIGN, "fp32 and int32 tensors must be 4-byte aligned");
    if (!a.lam) return da::fail(DA_ERR_NULL, "lam is NULL");
    if (a.nb > 0 && (!a.table || !a.bmap)) return da::fail(DA_ERR_NULL, "bias_table or bucket_map is NULL");
    if (static_cast<int64_t>(a.B) * a.rows == 0) return DA_OK;
    if (!a.q || !out) return da::fail(DA_ERR_NULL, "q or out is NULL");
    if (a.pg.num_pages > 0 && a.Lk > 0 && (!a.k || !a.v)) return da::fail(DA_ERR_NULL, "the cache is NULL");
    if (pl.total > 0) {
        if (!workspace || workspace_bytes < pl.total)
            return da::fail(DA_ERR_WORKSPACE, "workspace of %zu bytes; %zu are needed", workspace ? workspace_bytes : size_t{0}, pl.total);
        if (!da::aligned(workspace, 256)) return da::fail(DA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    }
    a.out = out;
    a.part_o = reinterpret_cast<float *>(static_cast<char *>(workspace) + pl.part_o);
    a.part_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) + pl.part_ml);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (pl.tensor) {
        pl.tc.slots = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + pl.slots);
        pl.tc.d = a;
        return p->dtype == DA_BF16 ? da::paged_forward_bf16(pl.tc, cs) : da::paged_forward_f16(pl.tc, cs);
    }
    cudaError_t e = pl.few ? da::paged_forward_few(a, p->dtype, pl.quads, cs) : da::paged_forward_general(a, p->dtype, cs);
    if (e == cudaSuccess && a.splits > 1) e = da::paged_merge(a, p->dtype, cs);
    return e == cudaSuccess ? DA_OK : da::cuda_fail(e, "paged attention launch");
}

}  // extern "C"
