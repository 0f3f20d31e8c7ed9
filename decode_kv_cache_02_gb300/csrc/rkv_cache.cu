// rkv_cache.cu -- the C ABI of the cache in use (declared in include/rkv.h):
// rotary plans, appends to paged and packed caches, and attention over them.
// Argument checks and the launch of k_tokens.cu and k_attention.cu; nothing
// here allocates or synchronises, and no state is kept between calls but on
// which devices an attention kernel's shared memory has been asked for (the
// runtime keeps that for every context of the device, also after a reset).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/rkv.h"
#include "rkv_common.cuh"
#include "rkv_internal.h"

namespace {

using rkv::AttnArgs;
using rkv::AttnPlan;
using rkv::DeviceStatus;
using rkv::RowsView;
using rkv::TokenArgs;

constexpr size_t kAlign = 256;
constexpr double kTwoPi = 6.283185307179586476925286766559;
// heads of a token: bounds the work items of a block to 32 bits
constexpr int64_t kMaxHeads = 16384;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_ws(const void* p) { return (reinterpret_cast<uintptr_t>(p) % kAlign) == 0; }
int64_t elem(int dtype) { return dtype == RKV_DTYPE_BF16 ? 2 : 4; }

// A byte range [lo, hi) of memory.
struct Span {
    uintptr_t lo = 0, hi = 0;
};
bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
Span span_of(const void* p, int64_t bytes) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return Span{b, b + (uintptr_t)bytes};
}

// Checks rows of `heads` heads: pointer and strides a multiple of 16 bytes,
// strides not negative (and, written to, rows that do not meet).  seqs x
// per_seq tokens, or (seqs 1) tokens numbered through.
int check_rows(const rkv_rows* r, int dtype, int d, int64_t heads, int64_t seqs, int64_t per_seq,
               bool written, RowsView* v, Span* span) {
    if (!r || !r->data || !aligned16(r->data)) return RKV_ERR_INVALID_ARG;
    const int64_t es = elem(dtype), unit = 16 / es;
    const int64_t st[3] = {seqs > 1 ? r->seq_stride : 0, per_seq > 1 ? r->token_stride : 0,
                           heads > 1 ? r->head_stride : 0};
    const int64_t n[3] = {seqs, per_seq, heads};
    int64_t last = d;
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0 || st[i] % unit != 0 || st[i] > ((int64_t)1 << 40)) return RKV_ERR_INVALID_ARG;
        last += st[i] * (n[i] > 0 ? n[i] - 1 : 0);
    }
    if (written) {
        // sorted by stride, each step passes all that lies within it
        int o[3] = {0, 1, 2};
        for (int i = 0; i < 2; ++i)
            for (int k = 0; k < 2 - i; ++k)
                if (st[o[k]] > st[o[k + 1]]) {
                    const int x = o[k];
                    o[k] = o[k + 1];
                    o[k + 1] = x;
                }
        int64_t extent = d;
        for (int i = 0; i < 3; ++i) {
            if (n[o[i]] <= 1) continue;
            if (st[o[i]] < extent) return RKV_ERR_INVALID_ARG;
            extent = st[o[i]] * (n[o[i]] - 1) + extent;
        }
    }
    v->data = r->data;
    v->seq = st[0];
    v->tok = st[1];
    v->head = st[2];
    v->heads = (int)heads;
    *span = span_of(r->data, last * es);
    return RKV_OK;
}

// Whether rows a (written in place) stay clear of rows b of the same tokens:
// memory apart, or two slices of the rows of one projection.
bool apart(const RowsView& a, const Span& as, const RowsView& b, const Span& bs, int dtype, int d,
           int64_t seqs, int64_t per_seq) {
    if (!overlap(as, bs)) return true;
    if (a.tok != b.tok || a.seq != b.seq) return false;
    const int64_t es = elem(dtype);
    const int64_t wa = (int64_t)(a.heads - 1) * a.head + d, wb = (int64_t)(b.heads - 1) * b.head + d;
    const bool first = as.lo <= bs.lo;
    const int64_t off = (int64_t)(first ? bs.lo - as.lo : as.lo - bs.lo) / es;
    // side by side within a token's row, the next token (whichever of tokens and
    // sequences are neighbours) behind both, and the next row of those behind all
    if (off < (first ? wa : wb)) return false;
    int64_t width = off + (first ? wb : wa);
    int64_t st[2] = {a.tok, a.seq}, n[2] = {per_seq, seqs};
    if (n[0] > 1 && n[1] > 1 && st[0] > st[1]) {
        st[0] = a.seq; st[1] = a.tok;
        n[0] = seqs; n[1] = per_seq;
    }
    for (int i = 0; i < 2; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < width) return false;
        width += st[i] * (n[i] - 1);
    }
    return true;
}

bool same_rows(const RowsView& a, const RowsView& b) {
    return a.data == b.data && a.seq == b.seq && a.tok == b.tok && a.head == b.head;
}

int check_plan(const rkv_rope_plan* p, int head_dim) {
    if (p->rot_dim < 2 || p->rot_dim > head_dim || (p->rot_dim & 1) != 0 ||
        (p->interleaved != 0 && p->interleaved != 1) || !isfinite(p->attn_factor))
        return RKV_ERR_INVALID_ARG;
    return RKV_OK;
}

void use_plan(const rkv_rope_plan* p, TokenArgs* a) {
    a->rot = p->rot_dim;
    a->interleaved = p->interleaved;
    a->factor = p->attn_factor;
    memcpy(a->turns, p->turns, sizeof(a->turns));
}

int rc_of(cudaError_t e) { return e == cudaSuccess ? RKV_OK : RKV_ERR_CUDA; }

cudaError_t run_tokens(const void* a, cudaStream_t s) {
    return rkv::launch_tokens(*static_cast<const TokenArgs*>(a), s);
}

int64_t pool_rows(const rkv_paged_desc* d) {
    return (int64_t)d->num_blocks * d->num_kv_heads * d->block_size;
}

// The part of an append that does not depend on the cache's format.
int check_append(const rkv_paged_desc* desc, const rkv_rope_plan* rope, const int32_t* table,
                 const int32_t* lens, int64_t num_tokens, int new_per_seq,
                 const int32_t* cu_tokens, const int32_t* positions, const rkv_rows* k,
                 const rkv_rows* v, const rkv_rows* q, const rkv_rows* out_q, void* workspace,
                 TokenArgs* a, Span* out_span, Span (&in)[3]) {
    int rc = rkv::check_paged_call(desc, table, &a->pg);
    if (rc) return rc;
    if (num_tokens < 0 || num_tokens >= ((int64_t)1 << 31)) return RKV_ERR_INVALID_ARG;
    if (!cu_tokens && (new_per_seq < 0 || num_tokens != desc->num_seqs * (int64_t)new_per_seq))
        return RKV_ERR_INVALID_ARG;
    if ((int64_t)desc->num_kv_heads * desc->gqa_group > kMaxHeads) return RKV_ERR_UNSUPPORTED;
    if (rope && (rc = check_plan(rope, desc->head_dim))) return rc;
    if (workspace && !aligned_ws(workspace)) return RKV_ERR_WORKSPACE;
    a->num_tokens = num_tokens;
    if (num_tokens == 0 || desc->num_seqs == 0) {
        a->num_tokens = 0;
        return RKV_OK;
    }
    if (!table || !lens) return RKV_ERR_INVALID_ARG;
    a->dtype = desc->dtype;
    a->d = desc->head_dim;
    a->num_seqs = desc->num_seqs;
    a->per_seq = cu_tokens ? num_tokens : new_per_seq;
    a->cu = cu_tokens;
    a->lens = lens;
    a->positions = positions;
    a->status = static_cast<DeviceStatus*>(workspace);
    if (rope) use_plan(rope, a);
    const int64_t seqs = num_tokens / a->per_seq;
    const int H = desc->num_kv_heads;
    if ((rc = check_rows(k, a->dtype, a->d, H, seqs, a->per_seq, false, &a->k, &in[0]))) return rc;
    if ((rc = check_rows(v, a->dtype, a->d, H, seqs, a->per_seq, false, &a->v, &in[1]))) return rc;
    if (q) {
        const int64_t Hq = (int64_t)H * desc->gqa_group;
        if ((rc = check_rows(q, a->dtype, a->d, Hq, seqs, a->per_seq, false, &a->q, &in[2])))
            return rc;
        if ((rc = check_rows(out_q, a->dtype, a->d, Hq, seqs, a->per_seq, true, &a->out_q, out_span)))
            return rc;
        // out_q is q itself, beside the k and v of a fused projection, or memory
        // of its own
        if (same_rows(a->q, a->out_q)) {
            if (!apart(a->q, in[2], a->k, in[0], a->dtype, a->d, seqs, a->per_seq) ||
                !apart(a->q, in[2], a->v, in[1], a->dtype, a->d, seqs, a->per_seq))
                return RKV_ERR_ALIAS;
        } else if (overlap(*out_span, in[0]) || overlap(*out_span, in[1]) ||
                   overlap(*out_span, in[2])) {
            return RKV_ERR_ALIAS;
        }
    } else if (out_q) {
        return RKV_ERR_INVALID_ARG;
    }
    return RKV_OK;
}

bool meets_any(const Span& pool, const Span& out, const Span (&in)[3]) {
    return overlap(pool, out) || overlap(pool, in[0]) || overlap(pool, in[1]) || overlap(pool, in[2]);
}

int check_q8(const rkv_paged_desc* d, const rkv_q8_cache* c, rkv::Q8Pools* p, Span (&spans)[4]) {
    if (!c) return RKV_ERR_INVALID_ARG;
    void* const at[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
    const int64_t rows = pool_rows(d);
    for (int i = 0; i < 4; ++i) {
        if (!at[i] || !aligned16(at[i])) return RKV_ERR_INVALID_ARG;
        spans[i] = span_of(at[i], rows * (i % 2 ? 4 : d->head_dim));
        for (int j = 0; j < i; ++j)
            if (overlap(spans[i], spans[j])) return RKV_ERR_ALIAS;
    }
    p->k_codes = static_cast<uint8_t*>(at[0]);
    p->k_scales = static_cast<float*>(at[1]);
    p->v_codes = static_cast<uint8_t*>(at[2]);
    p->v_scales = static_cast<float*>(at[3]);
    return RKV_OK;
}

int check_q4(const rkv_paged_desc* d, const rkv_q4_cache* c, rkv::Q4Pools* p, Span (&spans)[4]) {
    if (!c) return RKV_ERR_INVALID_ARG;
    void* const at[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
    const int64_t rows = pool_rows(d);
    for (int i = 0; i < 4; ++i) {
        if (!at[i] || !aligned16(at[i])) return RKV_ERR_INVALID_ARG;
        spans[i] = span_of(at[i], rows * (i % 2 ? d->head_dim / 8 : d->head_dim / 2));
        for (int j = 0; j < i; ++j)
            if (overlap(spans[i], spans[j])) return RKV_ERR_ALIAS;
    }
    p->k_codes = static_cast<uint8_t*>(at[0]);
    p->k_scales = static_cast<uint32_t*>(at[1]);
    p->v_codes = static_cast<uint8_t*>(at[2]);
    p->v_scales = static_cast<uint32_t*>(at[3]);
    return RKV_OK;
}

// The sizes of an attention call; the plan follows from them alone.
int check_attention(const rkv_paged_desc* desc, const int32_t* table, int n_new, int max_rows,
                    int bits, AttnArgs* a) {
    const int rc = rkv::check_paged_call(desc, table, &a->pg);
    if (rc) return rc;
    if (n_new < 1 || max_rows < 1 ||
        (int64_t)max_rows > (int64_t)desc->max_blocks_per_seq * desc->block_size)
        return RKV_ERR_INVALID_ARG;
    if (n_new > RKV_MAX_NEW_TOKENS || max_rows > (1 << 30) || (int64_t)desc->num_kv_heads * desc->gqa_group > kMaxHeads ||
        (bits && desc->dtype != RKV_DTYPE_BF16))
        return RKV_ERR_UNSUPPORTED;
    a->dtype = desc->dtype;
    a->d = desc->head_dim;
    a->G = desc->gqa_group;
    a->bits = bits;
    a->n_new = n_new;
    a->max_rows = max_rows;
    a->num_seqs = desc->num_seqs;
    return RKV_OK;
}

struct AttnCall {
    AttnArgs args;
    AttnPlan plan;
};
cudaError_t run_attention(const void* x, cudaStream_t s) {
    const AttnCall& c = *static_cast<const AttnCall*>(x);
    return rkv::launch_attention(c.args, c.plan, s);
}
cudaError_t run_combine(const void* x, cudaStream_t s) {
    const AttnCall& c = *static_cast<const AttnCall*>(x);
    return rkv::launch_attention_combine(c.args, c.plan, s);
}

size_t aligned_floats(size_t n) { return (n * sizeof(float) + kAlign - 1) / kAlign * kAlign; }
size_t attention_bytes(size_t scratch_floats) { return kAlign + aligned_floats(scratch_floats); }

// The parts of an attention call that do not depend on its workspace: pools, tables and
// rows.
int check_attend(const rkv_paged_desc* desc, int n_new, const rkv_rows* q, const void* K_pool,
                 const void* V_pool, const rkv_q4_cache* four, const rkv_q8_cache* eight,
                 const int32_t* table, const int32_t* lens, float scale, const rkv_rows* out,
                 float* lse, int bits, AttnArgs* a) {
    int rc;
    if (!table || !lens) return RKV_ERR_INVALID_ARG;
    const int64_t Hq = (int64_t)desc->num_kv_heads * desc->gqa_group;
    Span qs, os;
    if ((rc = check_rows(q, a->dtype, a->d, Hq, desc->num_seqs, n_new, false, &a->q, &qs))) return rc;
    if ((rc = check_rows(out, a->dtype, a->d, Hq, desc->num_seqs, n_new, true, &a->out, &os)))
        return rc;
    if (overlap(qs, os)) return RKV_ERR_ALIAS;
    if (bits) {
        Span spans[4];
        if ((rc = bits == 4 ? check_q4(desc, four, &a->q4p, spans) : check_q8(desc, eight, &a->q8p, spans)))
            return rc;
        for (const Span& sp : spans)
            if (overlap(sp, os)) return RKV_ERR_ALIAS;
    } else {
        if (!K_pool || !V_pool || !aligned16(K_pool) || !aligned16(V_pool))
            return RKV_ERR_INVALID_ARG;
        const int64_t bytes = pool_rows(desc) * a->d * elem(a->dtype);
        if (overlap(span_of(K_pool, bytes), os) || overlap(span_of(V_pool, bytes), os))
            return RKV_ERR_ALIAS;
        a->k = K_pool;
        a->v = V_pool;
    }
    a->lens = lens;
    a->scale = scale;
    a->lse = lse;
    return RKV_OK;
}

// Whether the kernels' 32-bit counts hold the units and pool rows of a call.
bool countable(const rkv_paged_desc* desc, const AttnArgs& a, const AttnPlan& pl) {
    return a.num_seqs * a.pg.H * ((int64_t)(a.max_rows - 1) / pl.unit + 1 + pl.lead) <
               ((int64_t)1 << 31) &&
           pool_rows(desc) < ((int64_t)1 << 32) - 1;
}

cudaError_t enqueue_attention(const AttnCall& call, cudaStream_t s) {
    const int bits = call.args.bits;
    cudaError_t e = rkv::timed_cache(bits == 8 ? rkv::kCacheAttnQ8 : (bits == 4 ? rkv::kCacheAttnQ4 : rkv::kCacheAttn),
                                     s, run_attention, &call);
    if (e == cudaSuccess && call.plan.join)
        e = rkv::timed_cache(rkv::kCacheAttnCombine, s, run_combine, &call);
    return e;
}

int attend(const rkv_paged_desc* desc, int n_new, const rkv_rows* q, const void* K_pool,
           const void* V_pool, const rkv_q4_cache* four, const rkv_q8_cache* eight, const int32_t* table,
           const int32_t* lens, int max_rows, float scale, const rkv_rows* out, float* lse,
           void* workspace, size_t workspace_bytes, void* stream, int bits) {
    AttnCall call;
    AttnArgs& a = call.args;
    int rc = check_attention(desc, table, n_new, max_rows, bits, &a);
    if (rc) return rc;
    if (!isfinite(scale)) return RKV_ERR_INVALID_ARG;
    call.plan = rkv::attn_plan(a);
    if (!countable(desc, a, call.plan)) return RKV_ERR_UNSUPPORTED;
    if (!workspace || !aligned_ws(workspace) || workspace_bytes < attention_bytes(call.plan.partial_floats))
        return RKV_ERR_WORKSPACE;
    if (desc->num_seqs == 0) return RKV_OK;
    if ((rc = check_attend(desc, n_new, q, K_pool, V_pool, four, eight, table, lens, scale, out, lse, bits, &a)))
        return rc;
    a.status = static_cast<DeviceStatus*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kAlign);
    return rc_of(enqueue_attention(call, static_cast<cudaStream_t>(stream)));
}

// --------------------------------------------------------------- prefixes --

struct PrefixCall {
    rkv::PrefixArgs args;
    AttnPlan own;
    rkv::PrefixPlan plan;
    size_t own_bytes() const { return attention_bytes(own.partial_floats); }
    // of calls with these sizes or smaller ones, whatever their blocks are
    size_t bytes() const {
        return attention_bytes(rkv::attn_most_floats(args.own)) + aligned_floats(plan.raw_floats) +
               aligned_floats(rkv::prefix_most_floats(args));
    }
};

// The sizes of a call over prefixes, its plans, and whether it can be counted.
int check_prefix(const rkv_paged_desc* desc, const int32_t* table, int n_new, int max_rows,
                 const rkv_prefixes* p, PrefixCall* c) {
    rkv::PrefixArgs& a = c->args;
    const int rc = check_attention(desc, table, n_new, max_rows, 0, &a.own);
    if (rc) return rc;
    if (!p || p->num_prefixes < 0) return RKV_ERR_INVALID_ARG;
    if (p->num_prefixes > 0 &&
        (p->max_blocks < 1 || p->max_rows < 1 ||
         (int64_t)p->max_rows > (int64_t)p->max_blocks * desc->block_size))
        return RKV_ERR_INVALID_ARG;
    if (p->num_prefixes > 0 && p->max_rows > (1 << 30)) return RKV_ERR_UNSUPPORTED;
    if (p->num_prefixes > 0 && !p->cu_seqs && desc->num_seqs % p->num_prefixes != 0)
        return RKV_ERR_INVALID_ARG;
    a.table = p->table;
    a.lens = p->lens;
    a.cu = p->num_prefixes > 0 ? p->cu_seqs : nullptr;
    a.num_prefixes = p->num_prefixes;
    a.max_blocks = p->num_prefixes > 0 ? p->max_blocks : 1;
    a.max_rows = p->num_prefixes > 0 ? p->max_rows : 1;
    // before the plans: every query in 32 bits
    if (desc->num_seqs * (int64_t)desc->num_kv_heads * desc->gqa_group * n_new >= ((int64_t)1 << 31) ||
        p->num_prefixes >= (1 << 24))
        return RKV_ERR_UNSUPPORTED;
    c->own = rkv::attn_plan(a.own);
    c->plan = rkv::prefix_plan(a);
    const int64_t most = ((int64_t)a.max_rows - 1) / c->plan.unit + 1 + c->plan.lead;
    if (!countable(desc, a.own, c->own) || c->plan.tiles * most >= ((int64_t)1 << 31))
        return RKV_ERR_UNSUPPORTED;
    return RKV_OK;
}

cudaError_t run_prefix(const void* x, cudaStream_t s) {
    const PrefixCall& c = *static_cast<const PrefixCall*>(x);
    return rkv::launch_prefix(c.args, c.plan, s);
}
cudaError_t run_prefix_join(const void* x, cudaStream_t s) {
    const PrefixCall& c = *static_cast<const PrefixCall*>(x);
    return rkv::launch_prefix_join(c.args, c.plan, s);
}

// Rows of a packed cache as values: the checks and the launch of both formats.
template <typename Args, typename Cache, typename Check>
int read_rows(const rkv_paged_desc* desc, const Cache* cache, const int32_t* block_table,
              const int32_t* lens, const int32_t* first, int n_rows, void* out_K, void* out_V,
              void* workspace, void* stream, Check check, rkv::CacheKernel kernel,
              cudaError_t (*launch)(const void*, cudaStream_t), Args* a) {
    int rc = rkv::check_paged_call(desc, block_table, &a->pg);
    if (rc) return rc;
    if (n_rows < 0) return RKV_ERR_INVALID_ARG;
    if (workspace && !aligned_ws(workspace)) return RKV_ERR_WORKSPACE;
    if (desc->num_seqs == 0 || n_rows == 0) return RKV_OK;
    if (!block_table || !lens || (!out_K && !out_V) || !aligned16(out_K) || !aligned16(out_V))
        return RKV_ERR_INVALID_ARG;
    Span pools[4];
    if ((rc = check(desc, cache, &a->p, pools))) return rc;
    a->dtype = desc->dtype;
    a->d = desc->head_dim;
    const int64_t rows = desc->num_seqs * (int64_t)desc->num_kv_heads * n_rows;
    if (rows >= ((int64_t)1 << 30)) return RKV_ERR_UNSUPPORTED;
    const int64_t bytes = rows * a->d * elem(a->dtype);
    const Span ks = span_of(out_K, out_K ? bytes : 0), vs = span_of(out_V, out_V ? bytes : 0);
    if (overlap(ks, vs)) return RKV_ERR_ALIAS;
    for (const Span& p : pools)
        if (overlap(p, ks) || overlap(p, vs)) return RKV_ERR_ALIAS;
    a->num_seqs = desc->num_seqs;
    a->lens = lens;
    a->first = first;
    a->n_rows = n_rows;
    a->out_k = out_K;
    a->out_v = out_V;
    a->status = static_cast<DeviceStatus*>(workspace);
    return rc_of(rkv::timed_cache(kernel, static_cast<cudaStream_t>(stream), launch, a));
}

}  // namespace

extern "C" {

int rkv_rope_init_freqs(int rot_dim, int interleaved, const double* freqs, double attn_factor,
                        rkv_rope_plan* plan) {
    if (!plan || !freqs || rot_dim < 2 || rot_dim > RKV_MAX_ROT_DIM || (rot_dim & 1) != 0 ||
        (interleaved != 0 && interleaved != 1) || !isfinite((float)attn_factor))
        return RKV_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; ++i)
        if (!isfinite(freqs[i])) return RKV_ERR_INVALID_ARG;
    rkv_rope_plan p;
    memset(&p, 0, sizeof(p));
    p.rot_dim = rot_dim;
    p.interleaved = interleaved;
    p.attn_factor = (float)attn_factor;
    for (int i = 0; i < rot_dim / 2; ++i) {
        // whole turns per position drop out: positions are whole numbers
        double t = freqs[i] / kTwoPi;
        t -= floor(t);
        const double u = ldexp(t, 64);
        p.turns[i] = u >= 18446744073709551616.0 ? 0u : (uint64_t)u;
    }
    *plan = p;
    return RKV_OK;
}

int rkv_rope_init(const rkv_rope_config* c, rkv_rope_plan* plan) {
    if (!c || !plan) return RKV_ERR_INVALID_ARG;
    const int r = c->rot_dim;
    if (r < 2 || r > RKV_MAX_ROT_DIM || (r & 1) != 0 || c->scaling < RKV_ROPE_NONE ||
        c->scaling > RKV_ROPE_BY_PARTS || !(c->base > 0.0) || !isfinite(c->base) ||
        !(c->factor > 0.0) || !isfinite(c->factor))
        return RKV_ERR_INVALID_ARG;
    if (c->scaling == RKV_ROPE_BY_PARTS &&
        (!(c->original_len > 0.0) || !isfinite(c->original_len) || !isfinite(c->low) ||
         !isfinite(c->high) || !(c->low < c->high)))
        return RKV_ERR_INVALID_ARG;
    double base = c->base;
    if (c->scaling == RKV_ROPE_NTK) {
        if (r == 2) return RKV_ERR_INVALID_ARG;  // the exponent has no value
        base *= pow(c->factor, r / (r - 2.0));
    }
    double f[RKV_MAX_ROT_DIM / 2];
    for (int i = 0; i < r / 2; ++i) {
        f[i] = pow(base, -2.0 * i / r);
        if (c->scaling == RKV_ROPE_LINEAR) f[i] /= c->factor;
        if (c->scaling == RKV_ROPE_BY_PARTS) {
            double g = (c->original_len * f[i] / kTwoPi - c->low) / (c->high - c->low);
            g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            f[i] *= g + (1.0 - g) / c->factor;
        }
    }
    return rkv_rope_init_freqs(r, c->interleaved, f, c->attn_factor, plan);
}

int rkv_rope_apply(const rkv_rope_plan* plan, int dtype, int head_dim, int64_t num_tokens,
                   int64_t tokens_per_seq, const int32_t* positions, int inverse, int q_heads,
                   const rkv_rows* q, const rkv_rows* out_q, int k_heads, const rkv_rows* k,
                   const rkv_rows* out_k, void* stream) {
    if (!plan) return RKV_ERR_INVALID_ARG;
    if (dtype != RKV_DTYPE_BF16 && dtype != RKV_DTYPE_FP32) return RKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return RKV_ERR_UNSUPPORTED;
    int rc = check_plan(plan, head_dim);
    if (rc) return rc;
    if (num_tokens < 0 || num_tokens >= ((int64_t)1 << 31) || q_heads < 1 || (k && k_heads < 1) ||
        (!k && out_k))
        return RKV_ERR_INVALID_ARG;
    if (q_heads > kMaxHeads || (k && k_heads > kMaxHeads)) return RKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return RKV_OK;
    if (tokens_per_seq < 1 || num_tokens % tokens_per_seq != 0 || !positions)
        return RKV_ERR_INVALID_ARG;
    TokenArgs a;
    a.dtype = dtype;
    a.d = head_dim;
    a.num_tokens = num_tokens;
    a.per_seq = tokens_per_seq;
    a.positions = positions;
    a.inverse = inverse != 0;
    use_plan(plan, &a);
    const int64_t seqs = num_tokens / tokens_per_seq;
    Span in[2], out[2];
    if ((rc = check_rows(q, dtype, head_dim, q_heads, seqs, tokens_per_seq, false, &a.q, &in[0])) ||
        (rc = check_rows(out_q, dtype, head_dim, q_heads, seqs, tokens_per_seq, true, &a.out_q,
                         &out[0])))
        return rc;
    const bool q_in = same_rows(a.q, a.out_q);
    if (!q_in && overlap(in[0], out[0])) return RKV_ERR_ALIAS;
    if (k) {
        if ((rc = check_rows(k, dtype, head_dim, k_heads, seqs, tokens_per_seq, false, &a.k, &in[1])) ||
            (rc = check_rows(out_k, dtype, head_dim, k_heads, seqs, tokens_per_seq, true, &a.out_k,
                             &out[1])))
            return rc;
        const bool k_in = same_rows(a.k, a.out_k);
        // rows in place may be slices of one projection; an output of its own
        // lies apart from everything else
        if (!k_in && (overlap(in[1], out[1]) || overlap(in[0], out[1]) || overlap(out[0], out[1])))
            return RKV_ERR_ALIAS;
        if (!q_in && (overlap(in[1], out[0]) || overlap(out[0], out[1]))) return RKV_ERR_ALIAS;
        if ((q_in || k_in) && !apart(a.q, in[0], a.k, in[1], dtype, head_dim, seqs, tokens_per_seq))
            return RKV_ERR_ALIAS;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return rc_of(rkv::timed_cache(rkv::kCacheRope, s, run_tokens, &a));
}

int rkv_paged_append(const rkv_paged_desc* desc, const rkv_rope_plan* rope, void* K_pool,
                     void* V_pool, const int32_t* block_table, const int32_t* lens,
                     int64_t num_tokens, int new_per_seq, const int32_t* cu_tokens,
                     const int32_t* positions, const rkv_rows* k, const rkv_rows* v,
                     const rkv_rows* q, const rkv_rows* out_q, void* workspace, void* stream) {
    TokenArgs a;
    Span out, in[3];
    int rc = check_append(desc, rope, block_table, lens, num_tokens, new_per_seq, cu_tokens,
                          positions, k, v, q, out_q, workspace, &a, &out, in);
    if (rc || a.num_tokens == 0) return rc;
    if (!K_pool || !V_pool || !aligned16(K_pool) || !aligned16(V_pool)) return RKV_ERR_INVALID_ARG;
    const int64_t bytes = pool_rows(desc) * a.d * elem(a.dtype);
    const Span kp = span_of(K_pool, bytes), vp = span_of(V_pool, bytes);
    if (overlap(kp, vp) || meets_any(kp, out, in) || meets_any(vp, out, in)) return RKV_ERR_ALIAS;
    a.k_pool = K_pool;
    a.v_pool = V_pool;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return rc_of(rkv::timed_cache(rkv::kCacheAppend, s, run_tokens, &a));
}

int rkv_q4_append(const rkv_paged_desc* desc, const rkv_rope_plan* rope,
                  const rkv_q4_cache* cache, const int32_t* block_table, const int32_t* lens,
                  int64_t num_tokens, int new_per_seq, const int32_t* cu_tokens,
                  const int32_t* positions, const rkv_rows* k, const rkv_rows* v,
                  const rkv_rows* q, const rkv_rows* out_q, void* workspace, void* stream) {
    TokenArgs a;
    Span out, in[3], pools[4];
    int rc = check_append(desc, rope, block_table, lens, num_tokens, new_per_seq, cu_tokens,
                          positions, k, v, q, out_q, workspace, &a, &out, in);
    if (rc || a.num_tokens == 0) return rc;
    if ((rc = check_q4(desc, cache, &a.q4p, pools))) return rc;
    for (const Span& p : pools)
        if (meets_any(p, out, in)) return RKV_ERR_ALIAS;
    a.bits = 4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return rc_of(rkv::timed_cache(rkv::kCacheQ4Append, s, run_tokens, &a));
}

int rkv_q8_append(const rkv_paged_desc* desc, const rkv_rope_plan* rope,
                  const rkv_q8_cache* cache, const int32_t* block_table, const int32_t* lens,
                  int64_t num_tokens, int new_per_seq, const int32_t* cu_tokens,
                  const int32_t* positions, const rkv_rows* k, const rkv_rows* v,
                  const rkv_rows* q, const rkv_rows* out_q, void* workspace, void* stream) {
    TokenArgs a;
    Span out, in[3], pools[4];
    int rc = check_append(desc, rope, block_table, lens, num_tokens, new_per_seq, cu_tokens,
                          positions, k, v, q, out_q, workspace, &a, &out, in);
    if (rc || a.num_tokens == 0) return rc;
    if ((rc = check_q8(desc, cache, &a.q8p, pools))) return rc;
    for (const Span& p : pools)
        if (meets_any(p, out, in)) return RKV_ERR_ALIAS;
    a.bits = 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return rc_of(rkv::timed_cache(rkv::kCacheQ8Append, s, run_tokens, &a));
}

int rkv_q4_read(const rkv_paged_desc* desc, const rkv_q4_cache* cache,
                const int32_t* block_table, const int32_t* lens, const int32_t* first,
                int n_rows, void* out_K, void* out_V, void* workspace, void* stream) {
    rkv::Q4ReadArgs a;
    return read_rows(desc, cache, block_table, lens, first, n_rows, out_K, out_V, workspace, stream,
                     check_q4, rkv::kCacheQ4Read,
                     [](const void* x, cudaStream_t st) {
                         return rkv::launch_q4_read(*static_cast<const rkv::Q4ReadArgs*>(x), st);
                     },
                     &a);
}

int rkv_q8_read(const rkv_paged_desc* desc, const rkv_q8_cache* cache,
                const int32_t* block_table, const int32_t* lens, const int32_t* first,
                int n_rows, void* out_K, void* out_V, void* workspace, void* stream) {
    rkv::Q8ReadArgs a;
    return read_rows(desc, cache, block_table, lens, first, n_rows, out_K, out_V, workspace, stream,
                     check_q8, rkv::kCacheQ8Read,
                     [](const void* x, cudaStream_t st) {
                         return rkv::launch_q8_read(*static_cast<const rkv::Q8ReadArgs*>(x), st);
                     },
                     &a);
}

size_t rkv_attention_workspace_size(const rkv_paged_desc* desc, int n_new, int max_rows) {
    // one size serves the pool and the packed caches
    AttnArgs a;
    if (check_attention(desc, nullptr, n_new, max_rows, 0, &a)) return 0;
    size_t n = attention_bytes(rkv::attn_most_floats(a));
    if (desc->dtype == RKV_DTYPE_BF16)
        for (const int bits : {4, 8}) {
            a.bits = bits;
            const size_t m = attention_bytes(rkv::attn_most_floats(a));
            if (m > n) n = m;
        }
    return n;
}

int rkv_paged_attention(const rkv_paged_desc* desc, int n_new, const rkv_rows* q,
                        const void* K_pool, const void* V_pool, const int32_t* block_table,
                        const int32_t* lens, int max_rows, float scale, const rkv_rows* out,
                        float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    return attend(desc, n_new, q, K_pool, V_pool, nullptr, nullptr, block_table, lens, max_rows, scale,
                  out, lse, workspace, workspace_bytes, stream, 0);
}

int rkv_q4_attention(const rkv_paged_desc* desc, int n_new, const rkv_rows* q,
                     const rkv_q4_cache* cache, const int32_t* block_table, const int32_t* lens,
                     int max_rows, float scale, const rkv_rows* out, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
    return attend(desc, n_new, q, nullptr, nullptr, cache, nullptr, block_table, lens, max_rows, scale,
                  out, lse, workspace, workspace_bytes, stream, 4);
}

int rkv_q8_attention(const rkv_paged_desc* desc, int n_new, const rkv_rows* q,
                     const rkv_q8_cache* cache, const int32_t* block_table, const int32_t* lens,
                     int max_rows, float scale, const rkv_rows* out, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
    return attend(desc, n_new, q, nullptr, nullptr, nullptr, cache, block_table, lens, max_rows, scale,
                  out, lse, workspace, workspace_bytes, stream, 8);
}

size_t rkv_prefix_attention_workspace_size(const rkv_paged_desc* desc, int n_new, int max_rows,
                                           const rkv_prefixes* prefixes) {
    PrefixCall c;
    return check_prefix(desc, nullptr, n_new, max_rows, prefixes, &c) ? 0 : c.bytes();
}

int rkv_prefix_attention(const rkv_paged_desc* desc, int n_new, const rkv_rows* q,
                         const void* K_pool, const void* V_pool, const rkv_prefixes* prefixes,
                         const int32_t* block_table, const int32_t* lens, int max_rows, float scale,
                         const rkv_rows* out, float* lse, void* workspace, size_t workspace_bytes,
                         void* stream) {
    PrefixCall c;
    int rc = check_prefix(desc, block_table, n_new, max_rows, prefixes, &c);
    if (rc) return rc;
    if (!isfinite(scale)) return RKV_ERR_INVALID_ARG;
    if (!workspace || !aligned_ws(workspace) || workspace_bytes < c.bytes()) return RKV_ERR_WORKSPACE;
    if (desc->num_seqs == 0) return RKV_OK;
    if (prefixes->num_prefixes > 0 && (!prefixes->table || !prefixes->lens)) return RKV_ERR_INVALID_ARG;
    AttnArgs& a = c.args.own;
    if ((rc = check_attend(desc, n_new, q, K_pool, V_pool, nullptr, nullptr, block_table, lens, scale, out,
                           lse, 0, &a)))
        return rc;
    char* const ws = static_cast<char*>(workspace);
    a.status = reinterpret_cast<DeviceStatus*>(ws);
    a.partial = reinterpret_cast<float*>(ws + kAlign);
    a.raw = reinterpret_cast<float*>(ws + c.own_bytes());
    a.raw_ml = a.raw + c.plan.raw_floats / (a.d + 2) * a.d;
    c.args.partial = reinterpret_cast<float*>(ws + c.own_bytes() + aligned_floats(c.plan.raw_floats));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AttnCall own;
    own.args = a;
    own.plan = c.own;
    cudaError_t e = enqueue_attention(own, s);
    if (e == cudaSuccess) e = rkv::timed_cache(rkv::kCachePrefix, s, run_prefix, &c);
    if (e == cudaSuccess) e = rkv::timed_cache(rkv::kCachePrefixJoin, s, run_prefix_join, &c);
    return rc_of(e);
}

}  // extern "C"
