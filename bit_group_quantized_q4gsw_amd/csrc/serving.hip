// C-ABI front end of the decoder serving calls: norm to int8 rows, the 4-bit key/value cache and
// attention over it.  As in api.hip, every check runs on the host before any HIP call.
#include "api_util.h"
#include "internal.h"
#include "kv_attention.h"

using namespace q4gsw;

namespace {

constexpr int64_t kMaxBlocks = 0x7FFFFFFF;
constexpr float kMinCap = 1e-30f, kMaxCap = 1e30f;   // 1 / cap and cap log2(e) stay normal

q4gsw_status check_cache_shape(const q4gsw_kv_cache* c) {
    if (!c) return Q4GSW_E_NULL;
    if (c->pages < 1 || c->pages > (int64_t(1) << 31) - 1 || c->page_size < kKvMinPage || c->page_size > kKvMaxPage ||
        (c->page_size & (c->page_size - 1)) != 0 || c->heads < 1 || c->heads > 65535 || !kv_dim_ok(c->dim) ||
        c->reserved != 0)
        return Q4GSW_E_SHAPE;
    return Q4GSW_OK;
}

// pages * heads * blocks * 36 dim < 2^31 * 2^16 * 2^7 * 2^14 may pass 64 bits: refused above 2^62
bool cache_bytes(const q4gsw_kv_cache* c, uint64_t* bytes) {
    const unsigned __int128 b = (unsigned __int128)c->pages * c->heads * (c->page_size / kKvTok) * kv_unit_bytes(c->dim);
    if (b > (uint64_t(1) << 62)) return false;
    *bytes = (uint64_t)b;
    return true;
}

q4gsw_status check_cache(const q4gsw_kv_cache* c, KvView* v, Range* r) {
    q4gsw_status st = check_cache_shape(c);
    if (st != Q4GSW_OK) return st;
    if (!c->data) return Q4GSW_E_NULL;
    uint64_t need = 0;
    if (!cache_bytes(c, &need)) return Q4GSW_E_SHAPE;
    if (c->bytes < need) return Q4GSW_E_BUFFER;
    if (reinterpret_cast<uintptr_t>(c->data) & 15u) return Q4GSW_E_ALIGN;
    v->data = static_cast<uint8_t*>(c->data);
    v->pages = c->pages;
    v->page_size = c->page_size;
    v->heads = c->heads;
    v->dim = c->dim;
    v->bpp_log2 = 0;
    while ((kKvTok << v->bpp_log2) < c->page_size) ++v->bpp_log2;
    *r = range_of(c->data, need);
    return Q4GSW_OK;
}

q4gsw_status check_seqs(const q4gsw_kv_seqs* s, KvSeqs* v) {
    if (!s) return Q4GSW_E_NULL;
    if (s->batch < 1 || s->batch > (1 << 20) || s->tokens < 0 || s->tokens > kMaxM || s->table_cols < 0 ||
        s->table_cols > (1 << 26) || s->table_ld < s->table_cols || s->table_ld > kMaxDim)
        return Q4GSW_E_SHAPE;
    if (!s->cu || !s->lens || (s->table_cols > 0 && !s->table)) return Q4GSW_E_NULL;
    *v = KvSeqs{s->table, s->table_ld, s->table_cols, s->cu, s->lens, s->batch, s->tokens};
    return Q4GSW_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Bytes of token rows `ld` elements apart, the last one `row` elements long.
uint64_t rows_extent(int64_t tokens, int64_t ld, int64_t row, int es) {
    return tokens == 0 ? 0 : ((uint64_t)(tokens - 1) * ld + row) * es;
}

// How an attention call runs.
struct AttnPlan {
    bool prompt;                 // kv_prompt, else kv_rows
    int waves;                   // per workgroup
    int row_tiles, splits, chunk;
    float us;                    // estimate
};

struct AttnSize {
    int heads, dim, batch, rows; // rows: new tokens times query heads of a cache head
    int64_t blocks;              // of 32 keys that some row may see
    float mean;                  // of them that a row sees
    bool prec;                   // kv_prompt keeps the remainders of keys and values
};

constexpr int kCus = 256;
constexpr int kFewRows = 32;     // never the kernel of many rows

void finish_plan(AttnPlan& p, const AttnSize& n, int64_t splits) {
    p.splits = (int)(splits < 1 ? 1 : splits);
    p.chunk = (int)((n.blocks + p.splits - 1) / p.splits);
    p.chunk += p.chunk & 1;
    // the join: its launch, and the partials written and read at some 4 TB/s
    p.us = p.splits > 1 ? 3.0f + 2e-6f * p.splits * n.batch * n.heads * n.rows * n.dim : 0.0f;
}

// Few rows.  The splits of the keys fill the workgroups that fit the GPU at once (32 sequences of
// 1024 .. 4096 tokens, 8 heads of 128: 3 splits 31.5 us, 8 splits 34.7; two of 131072: 48 splits 58
// us, 192 splits 73), but a split has 8 blocks, and 16 blocks are not split at all: the join's
// launch costs more (509 tokens, heads of 64: 6.6 us, 2 splits 8.5; four of 1024, heads of 128: 10.9 us,
// 4 splits 9.4).  Where that leaves long
// splits and few turns, unlike lengths end at unlike times, and shorter splits balance them (64
// sequences of 4096 .. 16384: 1 split 209 us, 8 splits 151).  Eight waves serve a grid of at most
// a workgroup per CU (509 tokens: 6.6 us against 7.1; 1024 workgroups of 512 tokens: 15.4 against 11.6).
AttnPlan plan_rows(const AttnSize& n) {
    AttnPlan p{};
    p.row_tiles = (n.rows + 15) / 16;
    const int64_t groups = (int64_t)n.batch * n.heads * p.row_tiles, fit = kCus * kv_rows_waves(n.dim);
    int64_t splits = 1;
    if (n.blocks > 16) {
        splits = fit / groups < n.blocks / 8 ? fit / groups : n.blocks / 8;
        if (splits < 1) splits = 1;
        if (n.blocks > 96 * splits && groups < 4 * fit) splits = (n.blocks + 63) / 64;
    }
    finish_plan(p, n, splits);
    p.waves = groups * p.splits <= kCus ? 8 : 4;
    p.us += 6.0f + (0.15f + 0.65f * n.dim / 128) * groups * n.mean / (4 * kCus);
    return p;
}

// Many rows: eight waves share a tile's unpacking where that still gives every CU a workgroup
// (wider heads have registers for one wave a SIMD).
AttnPlan plan_prompt(const AttnSize& n) {
    AttnPlan p{};
    p.prompt = true;
    p.waves = n.dim <= 128 && (int64_t)n.batch * n.heads * ((n.rows + 255) / 256) >= kCus ? 8 : 4;
    p.row_tiles = (n.rows + 32 * p.waves - 1) / (32 * p.waves);
    const int64_t groups = (int64_t)n.batch * n.heads * p.row_tiles;
    const int64_t fill = (kCus * 3 / 2 + groups - 1) / groups, most = (n.blocks + 15) / 16;
    finish_plan(p, n, fill < most ? fill : most);
    // 64 keys are a turn; a workgroup's own turns, and all turns over the CUs (two groups of four waves each)
    const float longest = (n.dim <= 128 ? 3.3f : 9.0f) * 0.5f * p.chunk;
    const float all = (1.0f + 1.6f * n.dim / 128) * 0.5f * groups * n.mean / (kCus * (p.waves == 8 ? 1 : 2));
    p.us += 8.0f + (n.prec ? 1.5f : 1.0f) * (longest > all ? longest : all);
    return p;
}

AttnSize attention_size(int heads, int dim, int batch, int hq, int max_new, int max_ctx, int window, int dtype) {
    AttnSize n{heads, dim, batch, max_new * (hq / heads), 0, 0.0f, dtype != kBF16};
    int64_t span = max_ctx;
    float mean = max_ctx > max_new ? max_ctx - 0.5f * max_new : 0.5f * max_ctx;
    if (window) {
        // the first row's window may begin and the last row's end inside a block
        if (window + (int64_t)max_new + 30 < span) span = window + (int64_t)max_new + 30;
        if (window + 32.0f < mean) mean = window + 32.0f;
    }
    n.blocks = (span + kKvTok - 1) / kKvTok;
    n.mean = mean / kKvTok;
    return n;
}

// Many rows share a tile's unpacking but take 64 keys in turn after turn, few rows spread over the
// GPU; which is faster is estimated from the keys a row sees, with the times of one turn and of one
// tile of 16 rows by 32 keys on the busy GPU (prompts of 32 / 8 heads of 128 from their beginning, few
// against many rows: 512 tokens 18 against 23 us, 1024 tokens 40 against 56, 2048 tokens 111 against
// 127, two of 2048 tokens 203 against 94; 1024 tokens behind 7000: 367 against 185).  Up to 32 rows
// never fill the workgroup of many.
AttnPlan plan_attention(const AttnSize& n, int kernel) {
    if (kernel == Q4GSW_KV_MANY_ROWS) return plan_prompt(n);
    const AttnPlan few = plan_rows(n);
    if (n.rows <= kFewRows || kernel == Q4GSW_KV_FEW_ROWS) return few;
    const AttnPlan many = plan_prompt(n);
    return many.us < few.us ? many : few;
}

uint64_t plan_workspace(const AttnPlan& p, int64_t tokens, int hq, int dim) {
    return p.splits > 1 ? (uint64_t)p.splits * tokens * hq * (dim + 2) * 4 : 0;
}

q4gsw_status check_attention(const q4gsw_kv_cache* c, int64_t batch, int64_t tokens, int32_t hq, int32_t max_new,
                             int32_t max_ctx) {
    if (batch < 1 || batch > (1 << 20) || tokens < 0 || tokens > kMaxM || hq < 1 || hq > (1 << 20) ||
        hq % c->heads != 0 || max_new < 1 || max_new > kMaxM || max_ctx < 0)
        return Q4GSW_E_SHAPE;
    if (tokens * hq > kMaxBlocks || (int64_t)max_new * (hq / c->heads) > kMaxBlocks / 2) return Q4GSW_E_SHAPE;
    return Q4GSW_OK;
}

q4gsw_status read_kernel(const q4gsw_kv_options* o, const q4gsw_kv_cache* c, int32_t hq, int32_t max_new, int* kernel) {
    *kernel = o ? o->kernel : Q4GSW_KV_ANY;
    if (!o) return Q4GSW_OK;
    if (o->reserved != 0) return Q4GSW_E_SHAPE;
    if (*kernel < Q4GSW_KV_ANY || *kernel > Q4GSW_KV_MANY_ROWS) return Q4GSW_E_ROUTE;
    if (*kernel == Q4GSW_KV_MANY_ROWS && (int64_t)max_new * (hq / c->heads) <= kFewRows) return Q4GSW_E_ROUTE;
    return Q4GSW_OK;
}

}  // namespace

extern "C" {

q4gsw_status q4gsw_rmsnorm_dq8ca(const void* x, int32_t x_dtype, const void* residual, const void* weight,
                                 int32_t r_dtype, int64_t M, int64_t K, float eps, void* h, void* rows,
                                 uint64_t rows_bytes, float* values, void* stream) {
    if (!x || !weight || !rows) return Q4GSW_E_NULL;
    if (M < 1 || M > kMaxM || K < 1 || K > kMaxDim || !finite_f(eps) || eps < 0) return Q4GSW_E_SHAPE;
    if (!act_dtype_ok(x_dtype) || !act_dtype_ok(r_dtype)) return Q4GSW_E_DTYPE;
    const uint64_t need = dq8ca_rows_total(M, K);
    if (rows_bytes < need) return Q4GSW_E_BUFFER;
    if (reinterpret_cast<uintptr_t>(rows) & 255u) return Q4GSW_E_ALIGN;
    const uint64_t n = (uint64_t)M * K;
    const Range ins[3] = {range_of(x, n * esize(x_dtype)), range_of(residual, residual ? n * esize(r_dtype) : 0),
                          range_of(weight, (uint64_t)K * esize(r_dtype))};
    const Range outs[3] = {range_of(h, h ? n * esize(r_dtype) : 0), range_of(rows, need), range_of(values, values ? n * 4 : 0)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 3; ++j) {
            if (i == 0 && j == 1 && h == residual) continue;      // the residual stream updated in place
            if (overlap(outs[i], ins[j])) return Q4GSW_E_ALIAS;
        }
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return Q4GSW_E_ALIAS;
    }
    return hip_status(launch_rmsnorm_dq8ca(x, x_dtype, residual, r_dtype, weight, M, K, eps, h, dq8ca_rows_at(rows, M, K),
                                           values, static_cast<hipStream_t>(stream)));
}

q4gsw_status q4gsw_kv_bytes(const q4gsw_kv_cache* c, uint64_t* bytes) {
    if (!bytes) return Q4GSW_E_NULL;
    const q4gsw_status st = check_cache_shape(c);
    if (st != Q4GSW_OK) return st;
    return cache_bytes(c, bytes) ? Q4GSW_OK : Q4GSW_E_SHAPE;
}

q4gsw_status q4gsw_kv_append(const q4gsw_kv_cache* c, const q4gsw_kv_seqs* s, const void* k, int64_t k_ld, const void* v,
                             int64_t v_ld, int32_t dtype, void* stream) {
    KvView cv;
    KvSeqs sv;
    Range cr;
    q4gsw_status st = check_cache(c, &cv, &cr);
    if (st != Q4GSW_OK) return st;
    if ((st = check_seqs(s, &sv)) != Q4GSW_OK) return st;
    if (!act_dtype_ok(dtype)) return Q4GSW_E_DTYPE;
    if (sv.tokens == 0) return Q4GSW_OK;
    if (!k || !v) return Q4GSW_E_NULL;
    const int64_t row = (int64_t)cv.heads * cv.dim;
    if (k_ld < row || v_ld < row || k_ld > kMaxDim || v_ld > kMaxDim) return Q4GSW_E_SHAPE;
    const int es = esize(dtype);
    if (!aligned16(k) || !aligned16(v) || (k_ld * es) % 16 != 0 || (v_ld * es) % 16 != 0) return Q4GSW_E_ALIGN;
    if (overlap(cr, range_of(k, rows_extent(sv.tokens, k_ld, row, es))) ||
        overlap(cr, range_of(v, rows_extent(sv.tokens, v_ld, row, es))))
        return Q4GSW_E_ALIAS;
    return hip_status(launch_kv_append(cv, sv, k, k_ld, v, v_ld, dtype, static_cast<hipStream_t>(stream)));
}

q4gsw_status q4gsw_kv_read(const q4gsw_kv_cache* c, const q4gsw_kv_seqs* s, float* k, float* v, void* stream) {
    KvView cv;
    KvSeqs sv;
    Range cr;
    q4gsw_status st = check_cache(c, &cv, &cr);
    if (st != Q4GSW_OK) return st;
    if ((st = check_seqs(s, &sv)) != Q4GSW_OK) return st;
    if (sv.tokens == 0) return Q4GSW_OK;
    if (!k || !v) return Q4GSW_E_NULL;
    if (!aligned16(k) || !aligned16(v)) return Q4GSW_E_ALIGN;
    const uint64_t n = (uint64_t)sv.tokens * cv.heads * cv.dim * 4;
    const Range kr = range_of(k, n), vr = range_of(v, n);
    if (overlap(kr, vr) || overlap(kr, cr) || overlap(vr, cr)) return Q4GSW_E_ALIAS;
    return hip_status(launch_kv_read(cv, sv, k, v, static_cast<hipStream_t>(stream)));
}

q4gsw_status q4gsw_kv_attention_workspace_bytes(const q4gsw_kv_cache* c, int32_t batch, int64_t tokens, int32_t hq,
                                                int32_t max_new, int32_t max_ctx, uint64_t* bytes) {
    if (!bytes) return Q4GSW_E_NULL;
    q4gsw_status st = check_cache_shape(c);
    if (st != Q4GSW_OK) return st;
    if ((st = check_attention(c, batch, tokens, hq, max_new, max_ctx)) != Q4GSW_OK) return st;
    // a window changes the span of keys, with which either plan's splits grow, and may change the plan
    const AttnSize n = attention_size(c->heads, c->dim, batch, hq, max_new, max_ctx, 0, kBF16);
    const uint64_t few = plan_workspace(plan_rows(n), tokens, hq, c->dim);
    const uint64_t many = n.rows <= kFewRows ? 0 : plan_workspace(plan_prompt(n), tokens, hq, c->dim);
    *bytes = few > many ? few : many;
    return Q4GSW_OK;
}

q4gsw_status q4gsw_kv_attention_plan(const q4gsw_kv_cache* c, int32_t batch, int64_t tokens, int32_t hq, int32_t max_new,
                                     int32_t max_ctx, int32_t window, int32_t dtype, const q4gsw_kv_options* opts,
                                     q4gsw_kv_plan_info* info) {
    if (!info) return Q4GSW_E_NULL;
    q4gsw_status st = check_cache_shape(c);
    if (st != Q4GSW_OK) return st;
    if ((st = check_attention(c, batch, tokens, hq, max_new, max_ctx)) != Q4GSW_OK) return st;
    if (window < 0) return Q4GSW_E_SHAPE;
    if (!act_dtype_ok(dtype)) return Q4GSW_E_DTYPE;
    int kernel = 0;
    if ((st = read_kernel(opts, c, hq, max_new, &kernel)) != Q4GSW_OK) return st;
    const AttnPlan p = plan_attention(attention_size(c->heads, c->dim, batch, hq, max_new, max_ctx, window, dtype), kernel);
    *info = q4gsw_kv_plan_info{p.prompt ? Q4GSW_KV_MANY_ROWS : Q4GSW_KV_FEW_ROWS, p.waves, p.splits};
    return Q4GSW_OK;
}

q4gsw_status q4gsw_kv_attention(const q4gsw_kv_cache* c, const q4gsw_kv_seqs* s, const void* q, int64_t q_ld,
                                int32_t dtype, int32_t hq, int32_t max_new, int32_t max_ctx, int32_t window,
                                float softcap, void* out, void* ws, uint64_t ws_bytes, void* stream) {
    return q4gsw_kv_attention_ex(c, s, q, q_ld, dtype, hq, max_new, max_ctx, window, softcap, out, ws, ws_bytes, nullptr,
                                 stream);
}

q4gsw_status q4gsw_kv_attention_ex(const q4gsw_kv_cache* c, const q4gsw_kv_seqs* s, const void* q, int64_t q_ld,
                                   int32_t dtype, int32_t hq, int32_t max_new, int32_t max_ctx, int32_t window,
                                   float softcap, void* out, void* ws, uint64_t ws_bytes, const q4gsw_kv_options* opts,
                                   void* stream) {
    KvAttnArgs a{};
    Range cr;
    q4gsw_status st = check_cache(c, &a.c, &cr);
    if (st != Q4GSW_OK) return st;
    if ((st = check_seqs(s, &a.sq)) != Q4GSW_OK) return st;
    if ((st = check_attention(c, s->batch, s->tokens, hq, max_new, max_ctx)) != Q4GSW_OK) return st;
    if (window < 0 || !(softcap == 0.0f || (softcap >= kMinCap && softcap <= kMaxCap))) return Q4GSW_E_SHAPE;
    if (!act_dtype_ok(dtype)) return Q4GSW_E_DTYPE;
    int kernel = 0;
    if ((st = read_kernel(opts, c, hq, max_new, &kernel)) != Q4GSW_OK) return st;
    if (s->tokens == 0) return Q4GSW_OK;
    if (!q || !out) return Q4GSW_E_NULL;
    const int64_t row = (int64_t)hq * c->dim;
    const int es = esize(dtype);
    if (q_ld < row || q_ld > kMaxDim) return Q4GSW_E_SHAPE;
    if (!aligned16(q) || !aligned16(out) || (q_ld * es) % 16 != 0) return Q4GSW_E_ALIGN;
    const AttnPlan p = plan_attention(attention_size(c->heads, c->dim, s->batch, hq, max_new, max_ctx, window, dtype),
                                      kernel);
    const uint64_t need = plan_workspace(p, s->tokens, hq, c->dim);
    if ((int64_t)p.splits * p.row_tiles > kMaxBlocks / ((int64_t)s->batch * c->heads)) return Q4GSW_E_SHAPE;
    if (!ws_ok(ws, ws_bytes, need)) return Q4GSW_E_WORKSPACE;
    const Range qr = range_of(q, rows_extent(s->tokens, q_ld, row, es));
    const Range orr = range_of(out, (uint64_t)s->tokens * row * es), sr = range_of(ws, need);
    if (overlap(orr, qr) || overlap(orr, cr) || overlap(sr, orr) || overlap(sr, qr) || overlap(sr, cr))
        return Q4GSW_E_ALIAS;
    a.q = q;
    a.q_ld = q_ld;
    a.dtype = dtype;
    a.out = out;
    a.part = static_cast<float*>(ws);
    a.ml = a.part + (uint64_t)p.splits * s->tokens * row;
    a.hq = hq;
    a.group = hq / c->heads;
    a.max_new = max_new;
    a.window = window;
    a.cap_in = softcap > 0 ? 1.0f / softcap : 0.0f;
    a.cap_out = softcap * kLog2e;
    a.scale = 1.0f / __builtin_sqrtf((float)c->dim);
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.row_tiles = p.row_tiles;
    hipStream_t st_ = static_cast<hipStream_t>(stream);
    hipError_t e = p.prompt ? launch_kv_prompt(a, p.waves, st_) : launch_kv_rows(a, p.waves, st_);
    if (e == hipSuccess && p.splits > 1) e = launch_kv_join(a, st_);
    return hip_status(e);
}

}  // extern "C"
