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
    int r, waves;                // kv_rows: tiles of 16 r rows; waves per workgroup
    int row_tiles, splits, chunk;
    uint64_t ws_bytes;
};

// The splits grow with the span of keys, so a window never needs more workspace than the plan
// without one.
AttnPlan plan_attention(int heads, int dim, int batch, int64_t tokens, int hq, int max_new, int max_ctx, int window) {
    AttnPlan p{};
    const int64_t rows = (int64_t)max_new * (hq / heads);
    int64_t span = max_ctx;
    if (window && window + (int64_t)max_new + 63 < span) span = window + (int64_t)max_new + 63;
    const int64_t blocks = (span + kKvTok - 1) / kKvTok;
    p.prompt = rows > 64;
    int64_t want, most;
    if (p.prompt) {
        p.waves = dim <= 128 && (int64_t)batch * heads * ((rows + 255) / 256) >= 256 ? 8 : 4;
        p.row_tiles = (int)((rows + 32 * p.waves - 1) / (32 * p.waves));
        const int64_t pairs = (int64_t)batch * heads * p.row_tiles;
        want = (384 + pairs - 1) / pairs;
        most = (blocks + 15) / 16;
    } else {
        p.r = rows > 16 && dim <= 128 ? 2 : 1;
        p.row_tiles = (int)((rows + 16 * p.r - 1) / (16 * p.r));
        const int64_t pairs = (int64_t)batch * heads * p.row_tiles;
        p.waves = blocks <= 16 && dim <= 128 ? 8 : 4;
        want = (3072 + pairs - 1) / pairs;
        most = (blocks + 15) / 16;
    }
    p.splits = (int)(want < most ? want : most);
    if (p.splits < 1) p.splits = 1;
    p.ws_bytes = p.splits > 1 ? (uint64_t)p.splits * tokens * hq * (dim + 2) * 4 : 0;
    p.chunk = (int)((blocks + p.splits - 1) / p.splits);
    p.chunk += p.chunk & 1;
    return p;
}

q4gsw_status check_attention(const q4gsw_kv_cache* c, int64_t batch, int64_t tokens, int32_t hq, int32_t max_new,
                             int32_t max_ctx) {
    if (batch < 1 || batch > (1 << 20) || tokens < 0 || tokens > kMaxM || hq < 1 || hq > (1 << 20) ||
        hq % c->heads != 0 || max_new < 1 || max_new > kMaxM || max_ctx < 0)
        return Q4GSW_E_SHAPE;
    if (tokens * hq > kMaxBlocks || (int64_t)max_new * (hq / c->heads) > kMaxBlocks / 2) return Q4GSW_E_SHAPE;
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
    *bytes = plan_attention(c->heads, c->dim, batch, tokens, hq, max_new, max_ctx, 0).ws_bytes;
    return Q4GSW_OK;
}

q4gsw_status q4gsw_kv_attention(const q4gsw_kv_cache* c, const q4gsw_kv_seqs* s, const void* q, int64_t q_ld,
                                int32_t dtype, int32_t hq, int32_t max_new, int32_t max_ctx, int32_t window,
                                float softcap, void* out, void* ws, uint64_t ws_bytes, void* stream) {
    KvAttnArgs a{};
    Range cr;
    q4gsw_status st = check_cache(c, &a.c, &cr);
    if (st != Q4GSW_OK) return st;
    if ((st = check_seqs(s, &a.sq)) != Q4GSW_OK) return st;
    if ((st = check_attention(c, s->batch, s->tokens, hq, max_new, max_ctx)) != Q4GSW_OK) return st;
    if (window < 0 || !(softcap == 0.0f || (softcap >= kMinCap && softcap <= kMaxCap))) return Q4GSW_E_SHAPE;
    if (!act_dtype_ok(dtype)) return Q4GSW_E_DTYPE;
    if (s->tokens == 0) return Q4GSW_OK;
    if (!q || !out) return Q4GSW_E_NULL;
    const int64_t row = (int64_t)hq * c->dim;
    const int es = esize(dtype);
    if (q_ld < row || q_ld > kMaxDim) return Q4GSW_E_SHAPE;
    if (!aligned16(q) || !aligned16(out) || (q_ld * es) % 16 != 0) return Q4GSW_E_ALIGN;
    const AttnPlan p = plan_attention(c->heads, c->dim, s->batch, s->tokens, hq, max_new, max_ctx, window);
    if ((int64_t)p.splits * p.row_tiles > kMaxBlocks / ((int64_t)s->batch * c->heads)) return Q4GSW_E_SHAPE;
    if (!ws_ok(ws, ws_bytes, p.ws_bytes)) return Q4GSW_E_WORKSPACE;
    const Range qr = range_of(q, rows_extent(s->tokens, q_ld, row, es));
    const Range orr = range_of(out, (uint64_t)s->tokens * row * es), sr = range_of(ws, p.ws_bytes);
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
    hipError_t e = p.prompt ? launch_kv_prompt(a, p.waves, st_) : launch_kv_rows(a, p.r, p.waves, st_);
    if (e == hipSuccess && p.splits > 1) e = launch_kv_join(a, st_);
    return hip_status(e);
}

}  // extern "C"
