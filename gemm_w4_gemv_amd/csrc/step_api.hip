// C ABI of the decode step's operators (w4_step.h): host-side validation and
// dispatch.  As in w4_api.hip, every check runs before the first HIP call.  An
// array without elements may have no address.
#include <math.h>

#include <initializer_list>

#include "kv4.hpp"
#include "w4_check.hpp"
#include "w4_step.h"

namespace {

using w4::aligned;
using w4::fail;
using w4::hip_fail;
using w4::overlap;
using w4::Range;
using w4::range;

bool any_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range& o : outs)
        for (const Range& i : ins)
            if (overlap(o, i)) return true;
    return false;
}
bool any_overlap(std::initializer_list<Range> outs) {
    for (const Range& a : outs)
        for (const Range& b : outs)
            if (&a != &b && overlap(a, b)) return true;
    return false;
}

// Bytes from the first to past the last value of ``rows`` rows of ``wide`` BF16.
Range rows_range(const void* p, int64_t rows, int64_t stride, int64_t wide) {
    return range(p, p && rows > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)wide) * 2 : 0);
}

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

struct CacheRanges {
    Range k, km, v, vm;
};
CacheRanges ranges_of(const w4_kv4_cache& c) {
    const size_t rows = (size_t)c.num_blocks * c.kv_heads * c.block_size;
    const size_t codes = rows * (c.head_dim / 2);
    const size_t meta = rows * (c.head_dim < W4_KV4_GROUP ? 1 : c.head_dim / W4_KV4_GROUP) * 4;
    return {range(c.k_codes, codes), range(c.k_meta, meta), range(c.v_codes, codes), range(c.v_meta, meta)};
}

w4_status check_cache(const char* fn, const w4_kv4_cache* c) {
    if (!c) return fail(W4_ERR_NULL, "%s: cache must not be NULL", fn);
    if (!c->k_codes || !c->k_meta || !c->v_codes || !c->v_meta)
        return fail(W4_ERR_NULL, "%s: the cache's arrays must not be NULL", fn);
    if (!head_dim_ok(c->head_dim))
        return fail(W4_ERR_UNSUPPORTED, "%s: head_dim %d (64, 128 and 256 are supported)", fn, c->head_dim);
    const int bs = c->block_size;
    if (bs < W4_KV4_MIN_BLOCK || bs > W4_KV4_MAX_BLOCK || (bs & (bs - 1)))
        return fail(W4_ERR_UNSUPPORTED, "%s: block_size %d (16, 32, 64, 128 and 256 are supported)", fn, bs);
    if (c->num_blocks < 1 || c->kv_heads < 1)
        return fail(W4_ERR_SHAPE, "%s: num_blocks = %d, kv_heads = %d must be at least 1", fn, c->num_blocks, c->kv_heads);
    if ((int64_t)c->num_blocks * bs > 0x7FFFFFFFll)
        return fail(W4_ERR_SHAPE, "%s: %d pages of %d slots: slots are 32-bit", fn, c->num_blocks, bs);
    if (!aligned(c->k_codes, 16) || !aligned(c->k_meta, 16) || !aligned(c->v_codes, 16) || !aligned(c->v_meta, 16))
        return fail(W4_ERR_ALIGN, "%s: the cache's arrays must be 16-byte aligned", fn);
    return W4_OK;
}

// A kernel launch counts its workgroups in 32 bits, and its work-items too.
constexpr int64_t kMaxGrid = 0x7FFFFFFFll;
constexpr int64_t kMaxItems = 0xFFFFFFFFll;

// Shared by w4_kv4_attn and its workspace size: the arguments that decide the split.
w4_status check_attn_shape(const char* fn, const w4_attn_args* a, const w4_kv4_cache* c) {
    if (!a || !c) return fail(W4_ERR_NULL, "%s: args and cache must not be NULL", fn);
    if (!head_dim_ok(c->head_dim))
        return fail(W4_ERR_UNSUPPORTED, "%s: head_dim %d (64, 128 and 256 are supported)", fn, c->head_dim);
    if (a->T < 0 || a->B < 0 || a->max_q < 0 || a->max_kv < 0 || a->q_heads < 1 || c->kv_heads < 1)
        return fail(W4_ERR_SHAPE, "%s: negative or zero size", fn);
    if (a->q_heads % c->kv_heads)
        return fail(W4_ERR_SHAPE, "%s: %d query heads are no multiple of %d key/value heads", fn, a->q_heads, c->kv_heads);
    if (a->window < 0 || a->sinks < 0) return fail(W4_ERR_ARG, "%s: window and sinks must not be negative", fn);
    const int64_t rows = (int64_t)a->max_q * a->q_heads;
    // workgroups of 256 threads, 16 rows of a key/value head each at least
    if (rows > (1ll << 28) || (int64_t)a->B * (rows / 16 + c->kv_heads) > kMaxGrid / 256)
        return fail(W4_ERR_SHAPE, "%s: %d requests of %d rows of %d heads are too many for one call", fn, a->B, a->max_q,
                    a->q_heads);
    return W4_OK;
}

}  // namespace

extern "C" {

W4_API w4_status w4_kv4_plan(const int32_t* cached, const int32_t* new_tokens, int32_t* block_table,
                             const int32_t* free_blocks, const int32_t* free_count, int B, int max_blocks,
                             int free_capacity, int block_size, int rows, int32_t* q_start, int32_t* kv_lens,
                             int32_t* positions, int32_t* slots, int32_t* counts, void* stream) {
    const char* fn = "w4_kv4_plan";
    if (B < 0 || max_blocks < 0 || free_capacity < 0 || rows < 0) return fail(W4_ERR_SHAPE, "%s: negative size", fn);
    if (!free_count || !q_start || !counts) return fail(W4_ERR_NULL, "%s: free_count, q_start and counts must not be NULL", fn);
    if (B > 0 && (!cached || !new_tokens || !kv_lens)) return fail(W4_ERR_NULL, "%s: cached, new_tokens and kv_lens must not be NULL", fn);
    if (B > 0 && max_blocks > 0 && !block_table) return fail(W4_ERR_NULL, "%s: block_table must not be NULL", fn);
    if (free_capacity > 0 && !free_blocks) return fail(W4_ERR_NULL, "%s: free_blocks must not be NULL", fn);
    if (rows > 0 && (!positions || !slots)) return fail(W4_ERR_NULL, "%s: positions and slots must not be NULL", fn);
    if (B > W4_KV4_PLAN_MAX_BATCH) return fail(W4_ERR_SHAPE, "%s: B = %d exceeds the limit %d", fn, B, W4_KV4_PLAN_MAX_BATCH);
    if ((int64_t)B * max_blocks > 0x7FFFFFFFll) return fail(W4_ERR_SHAPE, "%s: B * max_blocks exceeds 2^31 - 1", fn);
    if (block_size < 1 || block_size > 4096 || (block_size & (block_size - 1)))
        return fail(W4_ERR_ARG, "%s: block_size %d is no power of two in [1, 4096]", fn, block_size);
    for (const void* p : {(const void*)cached, (const void*)new_tokens, (const void*)block_table, (const void*)free_blocks,
                          (const void*)free_count, (const void*)q_start, (const void*)kv_lens, (const void*)positions,
                          (const void*)slots, (const void*)counts})
        if (!aligned(p, 4)) return fail(W4_ERR_ALIGN, "%s: arrays must be 4-byte aligned", fn);
    const Range rc = range(cached, (size_t)B * 4), rn = range(new_tokens, (size_t)B * 4),
                rt = range(block_table, (size_t)B * max_blocks * 4), rf = range(free_blocks, (size_t)free_capacity * 4),
                rk = range(free_count, 4), rq = range(q_start, ((size_t)B + 1) * 4), rl = range(kv_lens, (size_t)B * 4),
                rp = range(positions, (size_t)rows * 4), rs = range(slots, (size_t)rows * 4), ro = range(counts, 8);
    if (any_overlap({rt, rq, rl, rp, rs, ro}, {rc, rn, rf, rk}) || any_overlap({rt, rq, rl, rp, rs, ro}))
        return fail(W4_ERR_ALIAS, "%s: an output overlaps an input or another output", fn);
    const w4::PlanArgs a = {cached, new_tokens, block_table, free_blocks, free_count, B, max_blocks, free_capacity,
                            __builtin_ctz((unsigned)block_size), rows, q_start, kv_lens, positions, slots, counts};
    const hipError_t err = w4::launch_kv4_plan(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

W4_API w4_status w4_qk_norm_rope(const w4_qk_args* args, const w4_kv4_cache* cache, void* stream) {
    const char* fn = "w4_qk_norm_rope";
    if (!args) return fail(W4_ERR_NULL, "%s: args must not be NULL", fn);
    const w4_qk_args& a = *args;
    if (a.T < 0 || a.q_heads < 0 || a.kv_heads < 1) return fail(W4_ERR_SHAPE, "%s: T = %d, q_heads = %d, kv_heads = %d", fn, a.T, a.q_heads, a.kv_heads);
    if (!head_dim_ok(a.head_dim))
        return fail(W4_ERR_UNSUPPORTED, "%s: head_dim %d (64, 128 and 256 are supported)", fn, a.head_dim);
    if (a.q_heads > (1 << 16) || a.kv_heads > (1 << 16)) return fail(W4_ERR_SHAPE, "%s: more than 65536 heads", fn);
    if (a.rot_dim < 0 || a.rot_dim > a.head_dim || a.rot_dim % 16)
        return fail(W4_ERR_ARG, "%s: rot_dim = %d is no multiple of 16 in [0, head_dim]", fn, a.rot_dim);
    if (!(a.eps >= 0.0f) || !isfinite(a.eps) || !isfinite(a.weight_add))
        return fail(W4_ERR_ARG, "%s: eps must be finite and not negative, weight_add finite", fn);
    if (cache) {
        const w4_status st = check_cache(fn, cache);
        if (st != W4_OK) return st;
        if (cache->kv_heads != a.kv_heads || cache->head_dim != a.head_dim)
            return fail(W4_ERR_SHAPE, "%s: the cache has %d heads of %d, the call %d of %d", fn, cache->kv_heads,
                        cache->head_dim, a.kv_heads, a.head_dim);
        if (a.T > 0 && (!a.v || !a.slots)) return fail(W4_ERR_NULL, "%s: v and slots must not be NULL with a cache", fn);
    } else if (a.T > 0 && !a.k_out) {
        return fail(W4_ERR_NULL, "%s: k_out must not be NULL without a cache", fn);
    }
    if (a.T > 0 && (!a.k || (a.q_heads > 0 && (!a.q || !a.q_out))))
        return fail(W4_ERR_NULL, "%s: q, k and q_out must not be NULL", fn);
    if (a.rot_dim > 0) {
        if (!a.cos_sin || (a.T > 0 && !a.positions)) return fail(W4_ERR_NULL, "%s: cos_sin and positions must not be NULL", fn);
        if (a.max_pos < 1) return fail(W4_ERR_SHAPE, "%s: max_pos = %d must be at least 1", fn, a.max_pos);
    }
    if (a.T > 0 && w4::qk_norm_rope_groups(a, cache != nullptr) > kMaxItems / 256)
        return fail(W4_ERR_SHAPE, "%s: T = %d is too many rows for one call", fn, a.T);
    const int64_t qw = (int64_t)a.q_heads * a.head_dim, kw = (int64_t)a.kv_heads * a.head_dim;
    const auto stride_bad = [](int64_t s, int64_t wide) { return s < wide || s % 8 || s > (1ll << 40); };
    if ((a.q_heads > 0 && (stride_bad(a.q_stride, qw) || stride_bad(a.q_out_stride, qw))) || stride_bad(a.k_stride, kw) ||
        (cache && stride_bad(a.v_stride, kw)) || (a.k_out && stride_bad(a.k_out_stride, kw)))
        return fail(W4_ERR_ARG, "%s: row strides must be multiples of 8, at least heads * head_dim", fn);
    for (const void* p : {a.q, a.k, a.v, a.q_weight, a.k_weight, (const void*)a.cos_sin, (const void*)a.q_out, (const void*)a.k_out})
        if (!aligned(p, 16)) return fail(W4_ERR_ALIGN, "%s: q, k, v, weights, cos_sin and outputs must be 16-byte aligned", fn);
    if (!aligned(a.positions, 4) || !aligned(a.slots, 4)) return fail(W4_ERR_ALIGN, "%s: positions and slots must be 4-byte aligned", fn);
    const Range q = rows_range(a.q_heads ? a.q : nullptr, a.T, a.q_stride, qw), k = rows_range(a.k, a.T, a.k_stride, kw),
                v = rows_range(cache ? a.v : nullptr, a.T, a.v_stride, kw),
                qo = rows_range(a.q_heads ? a.q_out : nullptr, a.T, a.q_out_stride, qw),
                ko = rows_range(a.k_out, a.T, a.k_out_stride, kw),
                gq = range(a.q_weight, a.q_weight ? (size_t)a.head_dim * 2 : 0),
                gk = range(a.k_weight, a.k_weight ? (size_t)a.head_dim * 2 : 0),
                cs = range(a.cos_sin, a.rot_dim ? (size_t)a.max_pos * a.rot_dim * 4 : 0),
                po = range(a.positions, a.positions ? (size_t)a.T * 4 : 0), sl = range(a.slots, cache ? (size_t)a.T * 4 : 0);
    CacheRanges c = {};
    if (cache) c = ranges_of(*cache);
    // q, k and v may lie side by side in one buffer, and an output may be its
    // own input, so strided rows are told apart by their heads, not their span.
    const auto rows_apart = [&](const void* x, int64_t xs, int64_t xw, const void* y, int64_t ys, int64_t yw) {
        const Range rx = rows_range(x, a.T, xs, xw), ry = rows_range(y, a.T, ys, yw);
        if (!overlap(rx, ry)) return true;
        if (xs != ys || a.T < 1) return false;
        const int64_t step = xs * 2, d = (int64_t)(reinterpret_cast<uintptr_t>(y) - reinterpret_cast<uintptr_t>(x));
        const int64_t off = ((d % step) + step) % step;  // y's row begins so many bytes into x's
        return off >= xw * 2 && off + yw * 2 <= step;
    };
    const auto same = [](const void* x, int64_t xs, const void* y, int64_t ys) { return x == y && xs == ys; };
    const void* qi = a.q_heads ? a.q : nullptr;
    const void* qu = a.q_heads ? a.q_out : nullptr;
    const void* vi = cache ? a.v : nullptr;
    bool bad = false;
    if (qu && a.T > 0) {
        bad |= !same(qi, a.q_stride, qu, a.q_out_stride) && !rows_apart(qi, a.q_stride, qw, qu, a.q_out_stride, qw);
        bad |= !rows_apart(a.k, a.k_stride, kw, qu, a.q_out_stride, qw);
        bad |= vi && !rows_apart(vi, a.v_stride, kw, qu, a.q_out_stride, qw);
        bad |= a.k_out && !rows_apart(a.k_out, a.k_out_stride, kw, qu, a.q_out_stride, qw);
    }
    if (a.k_out && a.T > 0) {
        bad |= !same(a.k, a.k_stride, a.k_out, a.k_out_stride) && !rows_apart(a.k, a.k_stride, kw, a.k_out, a.k_out_stride, kw);
        bad |= qi && !rows_apart(qi, a.q_stride, qw, a.k_out, a.k_out_stride, kw);
        bad |= vi && !rows_apart(vi, a.v_stride, kw, a.k_out, a.k_out_stride, kw);
    }
    bad |= any_overlap({qo, ko, c.k, c.km, c.v, c.vm}, {gq, gk, cs, po, sl});
    bad |= any_overlap({c.k, c.km, c.v, c.vm}, {q, k, v, qo, ko}) || any_overlap({c.k, c.km, c.v, c.vm});
    if (bad) return fail(W4_ERR_ALIAS, "%s: an output overlaps an input or another output", fn);
    if (a.T == 0) return W4_OK;
    const hipError_t err = w4::launch_qk_norm_rope(a, cache, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

W4_API w4_status w4_kv4_read(const w4_kv4_cache* cache, const int32_t* slots, int n, void* k_out, void* v_out,
                             void* stream) {
    const char* fn = "w4_kv4_read";
    const w4_status st = check_cache(fn, cache);
    if (st != W4_OK) return st;
    if (n < 0) return fail(W4_ERR_SHAPE, "%s: n = %d is negative", fn, n);
    if (n > 0 && (!slots || (!k_out && !v_out))) return fail(W4_ERR_NULL, "%s: slots and one output must not be NULL", fn);
    if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return fail(W4_ERR_ALIGN, "%s: slots must be 4-byte, outputs 16-byte aligned", fn);
    if (w4::kv4_read_groups(*cache, n) > kMaxItems / 256) return fail(W4_ERR_SHAPE, "%s: n = %d is too many rows for one call", fn, n);
    const size_t bytes = (size_t)n * cache->kv_heads * cache->head_dim * 2;
    const Range ko = range(k_out, k_out ? bytes : 0), vo = range(v_out, v_out ? bytes : 0);
    const CacheRanges c = ranges_of(*cache);
    if (any_overlap({ko, vo}, {c.k, c.km, c.v, c.vm, range(slots, (size_t)n * 4)}) || overlap(ko, vo))
        return fail(W4_ERR_ALIAS, "%s: an output overlaps the cache, the slots or the other output", fn);
    if (n == 0) return W4_OK;
    const hipError_t err = w4::launch_kv4_read(*cache, slots, n, k_out, v_out, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

W4_API size_t w4_kv4_attn_workspace_bytes(const w4_attn_args* args, const w4_kv4_cache* cache) {
    if (check_attn_shape("w4_kv4_attn_workspace_bytes", args, cache) != W4_OK) return 0;
    if (args->T == 0 || args->B == 0 || args->max_q == 0) return 0;
    return w4::kv4_attn_workspace_bytes(*args, *cache);
}

W4_API w4_status w4_kv4_attn(const w4_attn_args* args, const w4_kv4_cache* cache, void* workspace,
                             size_t workspace_bytes, void* stream) {
    const char* fn = "w4_kv4_attn";
    if (!args) return fail(W4_ERR_NULL, "%s: args must not be NULL", fn);
    w4_status st = check_cache(fn, cache);
    if (st != W4_OK) return st;
    st = check_attn_shape(fn, args, cache);
    if (st != W4_OK) return st;
    const w4_attn_args& a = *args;
    if ((a.T > 0 && (!a.q || !a.out)) || (a.B > 0 && !a.kv_lens))
        return fail(W4_ERR_NULL, "%s: q, out and kv_lens must not be NULL", fn);
    if (a.max_blocks < 0) return fail(W4_ERR_SHAPE, "%s: max_blocks = %d is negative", fn, a.max_blocks);
    if (a.B > 0 && a.max_blocks > 0 && !a.block_table) return fail(W4_ERR_NULL, "%s: block_table must not be NULL", fn);
    if (!a.q_start && a.T != a.B) return fail(W4_ERR_SHAPE, "%s: without q_start T = %d must be B = %d", fn, a.T, a.B);
    if (!(a.scale > 0.0f) || !isfinite(a.scale)) return fail(W4_ERR_ARG, "%s: scale must be positive and finite", fn);
    const int64_t wide = (int64_t)a.q_heads * cache->head_dim;
    for (int64_t s : {a.q_stride, a.out_stride})
        if (s < wide || s % 8 || s > (1ll << 40))
            return fail(W4_ERR_ARG, "%s: row strides must be multiples of 8, at least q_heads * head_dim", fn);
    if (!aligned(a.q, 16) || !aligned(a.out, 16)) return fail(W4_ERR_ALIGN, "%s: q and out must be 16-byte aligned", fn);
    if (!aligned(a.block_table, 4) || !aligned(a.kv_lens, 4) || !aligned(a.q_start, 4))
        return fail(W4_ERR_ALIGN, "%s: block_table, kv_lens and q_start must be 4-byte aligned", fn);
    const size_t need = w4_kv4_attn_workspace_bytes(args, cache);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(W4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given%s", fn, need, workspace_bytes,
                        workspace ? "" : " (NULL)");
        if (!aligned(workspace, 16)) return fail(W4_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    }
    const Range q = rows_range(a.q, a.T, a.q_stride, wide), o = rows_range(a.out, a.T, a.out_stride, wide);
    const Range w = range(workspace, need), t = range(a.block_table, (size_t)a.B * a.max_blocks * 4),
                l = range(a.kv_lens, (size_t)a.B * 4), s = range(a.q_start, a.q_start ? ((size_t)a.B + 1) * 4 : 0);
    const CacheRanges c = ranges_of(*cache);
    if (any_overlap({o, w}, {q, t, l, s, c.k, c.km, c.v, c.vm}) || overlap(o, w))
        return fail(W4_ERR_ALIAS, "%s: out or workspace overlaps an input or each other", fn);
    if (a.T == 0 || a.B == 0 || a.max_q == 0) return W4_OK;
    const hipError_t err = w4::launch_kv4_attn(a, *cache, workspace, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

W4_API size_t w4_sample_workspace_bytes(int rows, int vocab) {
    if (rows <= 0 || vocab <= 0 || vocab > W4_SAMPLE_MAX_VOCAB) return 0;
    return w4::sample_workspace_bytes(rows, vocab);
}

W4_API w4_status w4_sample(const void* logits, int64_t row_stride, const double* uniform, const float* temperature,
                           const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens, int rows,
                           int vocab, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "w4_sample";
    if (rows != 0 && (!logits || !uniform || !tokens))
        return fail(W4_ERR_NULL, "%s: logits, uniform and tokens must not be NULL", fn);
    if (rows < 0 || rows > 65535) return fail(W4_ERR_SHAPE, "%s: rows = %d must lie in [0, 65535]", fn, rows);
    if (vocab < 1 || vocab > W4_SAMPLE_MAX_VOCAB)
        return fail(W4_ERR_SHAPE, "%s: vocab = %d must lie in [1, %d]", fn, vocab, W4_SAMPLE_MAX_VOCAB);
    if (row_stride < vocab || row_stride > (1ll << 40)) return fail(W4_ERR_ARG, "%s: row_stride is less than vocab", fn);
    if (!aligned(logits, 2) || !aligned(uniform, 8) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4))
        return fail(W4_ERR_ALIGN, "%s: logits must be 2-byte, uniform 8-byte, the others 4-byte aligned", fn);
    const size_t need = w4_sample_workspace_bytes(rows, vocab);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(W4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given%s", fn, need, workspace_bytes,
                        workspace ? "" : " (NULL)");
        if (!aligned(workspace, 16)) return fail(W4_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    }
    const size_t r4 = (size_t)rows * 4;
    const Range out = range(tokens, r4), w = range(workspace, need);
    if (any_overlap({out, w}, {rows_range(logits, rows, row_stride, vocab), range(uniform, 2 * r4),
                               range(temperature, temperature ? r4 : 0), range(top_k, top_k ? r4 : 0),
                               range(top_p, top_p ? r4 : 0), range(min_p, min_p ? r4 : 0)}) || overlap(out, w))
        return fail(W4_ERR_ALIAS, "%s: tokens or workspace overlaps an input or each other", fn);
    if (rows == 0) return W4_OK;
    const w4::SampleArgs a = {static_cast<const uint16_t*>(logits), row_stride, uniform, temperature, top_k, top_p,
                              min_p, tokens, rows, vocab};
    const hipError_t err = w4::launch_sample(a, workspace, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? W4_OK : hip_fail(err, fn);
}

}  // extern "C"
