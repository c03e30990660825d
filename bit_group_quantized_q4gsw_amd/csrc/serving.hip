// C-ABI front end of the decoder serving calls: norm to int8 rows, the 4-bit key/value cache and
// attention over it.  As in api.hip, every check runs on the host before any HIP call.
#include "api_util.h"
#include "internal.h"
#include "kv_attention.h"
#include "logits.h"

using namespace q4gsw;

namespace {

constexpr int64_t kMaxBlocks = 0x7FFFFFFF, kMaxThreads = 0xFFFFFFFF;
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

// Does an output overlap the arrays that describe the sequences?
bool over_seqs(const KvSeqs& s, Range out) {
    const uint64_t table = s.table_cols ? ((uint64_t)(s.batch - 1) * s.table_ld + s.table_cols) * 4 : 0;
    return overlap(out, range_of(s.table, table)) || overlap(out, range_of(s.cu, (uint64_t)(s.batch + 1) * 4)) ||
           overlap(out, range_of(s.lens, (uint64_t)s.batch * 4));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Bytes of token rows `ld` elements apart, the last one `row` elements long.
uint64_t rows_extent(int64_t tokens, int64_t ld, int64_t row, int es) {
    return tokens == 0 ? 0 : ((uint64_t)(tokens - 1) * ld + row) * es;
}

// How an attention call runs.
struct AttnPlan {
    enum { kRows, kTree, kPrompt } kernel;
    int waves;                   // per workgroup
    int row_tiles, splits, chunk;
    float us;                    // estimate
};

struct AttnSize {
    int heads, dim, batch, rows; // rows: new tokens times query heads of a cache head
    int group, max_new, max_ctx, window;
    float mean;                  // blocks of 32 keys that a row sees
    bool prec;                   // kv_prompt keeps the remainders of keys and values
    bool tree;                   // any node of a tree may be a root: its window begins at the first one's

    // Blocks that some tile of `tile` rows may see: behind a window those of the window and of the
    // tile's own tokens, and its first row's window may begin and its last row's end inside a block.
    int64_t blocks(int tile) const {
        int64_t span = max_ctx;
        if (window) {
            const int64_t own = tree ? max_new : (tile - 2) / group + 2, seen = window + (own < max_new ? own : max_new) + 30;
            span = seen < span ? seen : span;
        }
        return (span + kKvTok - 1) / kKvTok;
    }
};

constexpr int kCus = 256;
constexpr int kFewRows = 32;     // never the kernel of many rows

void finish_plan(AttnPlan& p, const AttnSize& n, int64_t blocks, int64_t splits) {
    p.splits = (int)(splits < 1 ? 1 : splits);
    p.chunk = (int)((blocks + p.splits - 1) / p.splits);
    p.chunk += p.chunk & 1;
    // the join: its launch, and the partials written and read at some 5 TB/s
    p.us = p.splits > 1 ? 3.0f + 1.6e-6f * p.splits * n.batch * n.heads * n.rows * n.dim : 0.0f;
}

// Few rows.  The splits of the keys fill the workgroups that fit the GPU at once (us, single tokens of 32 / 8
// heads of 128; 32 sequences of 1024 .. 4096 tokens, fp16: 3 splits 33, 1 split 38, 8 splits 34; two of 131072, bf16: 48
// splits 62, 192 splits 75), but a split has 8 blocks, and 16 blocks are not split at all: the join's
// launch costs more (509 tokens, heads of 64: 7.1, 2 splits 8.5; four of 1024: 11.7, 4 splits 9.7).  Where that leaves
// long splits and few turns, unlike lengths end at unlike times, and shorter splits balance them (64
// sequences of 4096 .. 16384: 1 split 207, 8 splits 171).  Eight waves serve a grid of at most a
// workgroup per CU (509 tokens: 7.1 against 7.7; 1024 workgroups of 512 tokens: 31.7 against 21.9).
// The estimate: time of a tile of 16 rows by 32 keys on a CU, of which a grid that fits at once gives the
// fullest CU a whole number, and of a workgroup's loads and join.
AttnPlan plan_rows(const AttnSize& n) {
    AttnPlan p{};
    p.row_tiles = (n.rows + 15) / 16;
    const int64_t groups = (int64_t)n.batch * n.heads * p.row_tiles, fit = kCus * kv_rows_waves(n.dim);
    const int64_t blocks = n.blocks(16);
    int64_t splits = 1;
    if (blocks > 16) {
        splits = fit / groups < blocks / 8 ? fit / groups : blocks / 8;
        if (splits < 1) splits = 1;
        if (blocks > 96 * splits && groups < 4 * fit) splits = (blocks + 63) / 64;
    }
    finish_plan(p, n, blocks, splits);
    p.waves = groups * p.splits <= kCus ? 8 : 4;
    const float turns = (float)groups * p.splits / fit;
    const float per_cu = turns <= 1 ? (float)((groups * p.splits + kCus - 1) / kCus) : (float)groups * p.splits / kCus;
    p.us += 2.5f + (0.09f + 0.0048f * n.dim) * per_cu * n.mean / (4 * p.splits) + (2.0f + 0.026f * n.dim) * (turns < 1 ? 1 : turns);
    return p;
}

// Trees, in tiles of 16 rows (kv_rows) or of 32 (kv_tree), `most` waves a workgroup, `unit` us that a CU takes for a unit
// of 32 keys and a tile.  VALU is the bound, so one workgroup of eight waves a CU does as well as more, and
// splits pay while they fill the CUs: us of 16 sequences of 1024 .. 4096 tokens, 32 / 8 heads of 128, bf16 (fp16), in
// tiles of 32, 8 nodes (128 workgroups): 1 split 38 (47), 2 splits 27 (32), 4 splits 28 (32), 8 splits 33 (40); 16
// nodes (256): 39 (47), 42 (51), 46 (56), 51 (65); 64 nodes (1024): 88 (117), 98 (128).  In tiles of 16, 8 sequences of
// 26 nodes, window 1024, 16 / 4 heads of 256 (224 workgroups): 1 split 24, 2 splits 32; up to 32 blocks none pay: 521
// tokens, heads of 64: 1 split 9.2, 2 splits 13.7.
// `waves`: what a SIMD holds; `start`: us of a workgroup's first loads, tree and join, which the next turn of workgroups pays
// again (43 sequences of 62 nodes and 103 tokens, 24 / 4 heads of 192, fp16, 4128 tiles of 16 rows: 78, estimate 73).
AttnPlan plan_tiles(const AttnSize& n, int tile, int most, int waves, float unit, float start) {
    AttnPlan p{};
    p.row_tiles = (n.rows + tile - 1) / tile;
    const int64_t groups = (int64_t)n.batch * n.heads * p.row_tiles, blocks = n.blocks(tile);
    int64_t splits = 1;
    if (blocks > 32) splits = kCus / groups < blocks / 8 ? kCus / groups : blocks / 8;
    finish_plan(p, n, blocks, splits);
    p.waves = groups * p.splits <= kCus ? most : 4;
    const int64_t all = groups * p.splits;
    const float turns = (float)all * p.waves / (kCus * 4 * waves);
    const float per_cu = turns <= 1 ? (float)((all + kCus - 1) / kCus) : (float)all / kCus;
    const float longest = (float)((p.chunk + p.waves - 1) / p.waves * p.waves), mean = per_cu * n.mean / p.splits;
    p.us += start * (turns < 1 ? 1 : turns) + unit * (longest > mean ? longest : mean);
    return p;
}

AttnPlan plan_tree(const AttnSize& n) {
    const float unit = n.dim <= 192 ? 0.04f + 0.0017f * n.dim : 0.6f;       // one wave a SIMD at 256 channels
    AttnPlan p = plan_tiles(n, 32, kv_tree_most(n.dim), kv_tree_waves(n.dim, n.prec), unit * (n.prec ? 1.25f : 1.0f), 4.5f + 0.035f * n.dim);
    p.kernel = AttnPlan::kTree;
    return p;
}

// us of a turn of 64 keys of a workgroup that fills its CU (eight waves up to 128 channels, four above).
float prompt_turn(int dim, bool prec) {
    if (dim <= 128) return prec ? 0.66f + 0.0235f * dim : 0.65f + 0.0135f * dim;
    return prec ? 0.8f + 0.0211f * dim : 0.47f + 0.013f * dim;
}

// Most splits of the kernel of many rows with `waves` a workgroup: of 16 blocks at least, and as many as
// keep every workgroup of the grid on the GPU at once.  One more launches a second turn of workgroups
// and halves what each has to do (32 / 8 heads of 128, bf16, `waves` 8: 2048 tokens, 256 workgroups: 74 us,
// 2 splits 106; 1024 behind 7000, 128 workgroups: 2 splits 161 us, 1 split 237, 3 splits 198).
int64_t prompt_splits(const AttnSize& n, int waves, bool prec) {
    const int64_t groups = (int64_t)n.batch * n.heads * ((n.rows + 32 * waves - 1) / (32 * waves));
    const int64_t fill = kCus * prompt_fit(n.dim, prec, waves) / groups, most = (n.blocks(32 * waves) + 15) / 16;
    const int64_t splits = fill < most ? fill : most;
    return splits < 1 ? 1 : splits;
}

// Many rows: eight waves (up to 128 channels), which share a tile's unpacking, or four, and keys split as far
// as the grid fits or not at all, by the estimate: a workgroup's loads and end each time that one starts on a
// CU, and its own turns, or all turns over the CUs.  Of workgroups of
// four waves that fit a CU twice two take 1.3 times the turn of one of eight waves, and one alone 0.85 times.  Prompts
// from their beginning have rows of unlike lengths, which splits balance badly (1024 tokens, 32 / 8 heads of 128, bf16: four
// waves 37.5 us, 2 splits 47; eight waves 41 and 45); few rows need them (256 tokens behind 3744: eight waves
// and 8 splits 46 us, 4 splits 53, 1 split 124).
AttnPlan plan_prompt(const AttnSize& n) {
    AttnPlan best{};
    for (int waves = n.dim <= 128 ? 8 : 4; waves >= 4; waves -= 4) {
        AttnPlan p{};
        p.kernel = AttnPlan::kPrompt;
        p.waves = waves;
        p.row_tiles = (n.rows + 32 * waves - 1) / (32 * waves);
        const int64_t groups = (int64_t)n.batch * n.heads * p.row_tiles, most = prompt_splits(n, waves, n.prec);
        const int fit = prompt_fit(n.dim, n.prec, waves);
        const bool half = waves == 4 && n.dim <= 128;
        for (int64_t splits = 1;; splits = most) {
            finish_plan(p, n, n.blocks(32 * waves), splits);
            float turns = (float)groups * p.splits / (kCus * fit), starts = turns < 1 ? 1 : turns;
            if (fit == 1) {                                          // a last turn may fill few CUs
                starts = (float)((groups * p.splits + kCus - 1) / kCus);
                turns = turns < 0.9f * starts ? 0.9f * starts : turns;
            }
            const float all = (half ? (fit == 2 ? 1.3f : 0.85f) : 1.0f) * turns * 0.5f * n.mean / p.splits;
            const float longest = (half ? 0.85f : 1.0f) * 0.5f * p.chunk;
            p.us += (4.6f + 0.026f * n.dim) * starts + prompt_turn(n.dim, n.prec) * (longest > all ? longest : all);
            if (best.waves == 0 || p.us < best.us) best = p;
            if (splits >= most) break;
        }
    }
    return best;
}

AttnSize attention_size(int heads, int dim, int batch, int hq, int max_new, int max_ctx, int window, int dtype, bool tree = false) {
    float mean = max_ctx > max_new ? max_ctx - 0.5f * max_new : 0.5f * max_ctx;
    if (window && window + 32.0f < mean) mean = window + 32.0f;
    return AttnSize{heads, dim, batch, max_new * (hq / heads), hq / heads, max_new, max_ctx, window, mean / kKvTok, dtype != kBF16, tree};
}

// Many rows share a tile's unpacking but take 64 keys in turn after turn, few rows spread over the GPU;
// which is faster is estimated.  us measured, few against many rows, in bf16 (in fp16; fp32 is within 3% of it), prompts
// from their beginning of 32 / 8 heads of 128: 512 tokens 19 / 23 (18 / 27), 1024 tokens 42 / 38 (42 / 48), 2048 tokens
// 118 / 71 (119 / 97), two of 2048 tokens 223 / 98 (219 / 137); 1024 tokens behind 7000 377 / 161 (372 / 234); of 16 / 4 heads
// of 256: 2048 tokens 129 / 127 (130 / 198), two of 2048 tokens 235 / 152 (231 / 234), three chunks of 2048 behind 6144
// 1732 / 1262 (1735 / 2026).  Of 378 prompts, chunks and drafts of random sizes, 104 of
// them windowed, it takes the slower kernel by over 10% for 12, by 31% at most.  Up to 32 rows never fill the workgroup of many.
AttnPlan plan_attention(const AttnSize& n, int kernel) {
    if (kernel == Q4GSW_KV_MANY_ROWS) return plan_prompt(n);
    if (kernel == Q4GSW_KV_TREE) return plan_tree(n);
    AttnPlan few = n.tree ? plan_tiles(n, 16, 8, kv_rows_waves(n.dim), 0.06f + 0.00105f * n.dim, 4.0f + 0.02f * n.dim) : plan_rows(n);
    if (kernel == Q4GSW_KV_FEW_ROWS) return few;
    // (of 140 drawn calls of 10 to 120 us the estimates take a kernel slower by over 10% for 6, by 42% at most)
    // a tree's tiles of 32 rows cost less VALU a row, tiles of 16 spread over more CUs and start sooner (us of 16 nodes of
    // 600 tokens, 32 / 8 heads of 128, bf16: 10.5 against 14.2; the batch of plan_tiles' comment, 8 nodes: 31 against 27, 32
    // nodes in fp16 77 and 81)
    if (n.tree && n.rows > 16) {
        const AttnPlan wide = plan_tree(n);
        if (wide.us < few.us) few = wide;
    }
    if (n.rows <= kFewRows) return few;
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

q4gsw_status read_kernel(const q4gsw_kv_options* o, const q4gsw_kv_cache* c, int32_t hq, int32_t max_new, bool tree, int* kernel) {
    *kernel = o ? o->kernel : Q4GSW_KV_ANY;
    if (!o) return Q4GSW_OK;
    if (o->reserved != 0) return Q4GSW_E_SHAPE;
    if (*kernel < Q4GSW_KV_ANY || *kernel > (tree ? Q4GSW_KV_TREE : Q4GSW_KV_MANY_ROWS)) return Q4GSW_E_ROUTE;
    if (*kernel == Q4GSW_KV_MANY_ROWS && (int64_t)max_new * (hq / c->heads) <= kFewRows) return Q4GSW_E_ROUTE;
    return Q4GSW_OK;
}

// kv_attention, or with `parents` attention of trees.
q4gsw_status attend(const q4gsw_kv_cache* c, const q4gsw_kv_seqs* s, const int32_t* parents, bool tree, const void* q,
                    int64_t q_ld, int32_t dtype, int32_t hq, int32_t max_new, int32_t max_ctx, int32_t window, float softcap,
                    void* out, void* ws, uint64_t ws_bytes, const q4gsw_kv_options* opts, void* stream) {
    KvAttnArgs a{};
    Range cr;
    q4gsw_status st = check_cache(c, &a.c, &cr);
    if (st != Q4GSW_OK) return st;
    if ((st = check_seqs(s, &a.sq)) != Q4GSW_OK) return st;
    if ((st = check_attention(c, s->batch, s->tokens, hq, max_new, max_ctx)) != Q4GSW_OK) return st;
    if (tree && max_new > kTreeMax) return Q4GSW_E_SHAPE;
    if (window < 0 || !(softcap == 0.0f || (softcap >= kMinCap && softcap <= kMaxCap))) return Q4GSW_E_SHAPE;
    if (!act_dtype_ok(dtype)) return Q4GSW_E_DTYPE;
    int kernel = 0;
    if ((st = read_kernel(opts, c, hq, max_new, tree, &kernel)) != Q4GSW_OK) return st;
    if (s->tokens == 0) return Q4GSW_OK;
    if (!q || !out || (tree && !parents)) return Q4GSW_E_NULL;
    const int64_t row = (int64_t)hq * c->dim;
    const int es = esize(dtype);
    if (q_ld < row || q_ld > kMaxDim) return Q4GSW_E_SHAPE;
    if (!aligned16(q) || !aligned16(out) || (q_ld * es) % 16 != 0) return Q4GSW_E_ALIGN;
    const AttnPlan p = plan_attention(attention_size(c->heads, c->dim, s->batch, hq, max_new, max_ctx, window, dtype, tree),
                                      kernel);
    const uint64_t need = plan_workspace(p, s->tokens, hq, c->dim);
    // a grid takes fewer than 2^32 threads in one dimension; the join has up to 256 a row
    if ((int64_t)p.splits * p.row_tiles > kMaxThreads / (64 * p.waves * ((int64_t)s->batch * c->heads)) ||
        (p.splits > 1 && s->tokens * hq > kMaxThreads / 256))
        return Q4GSW_E_SHAPE;
    if (!ws_ok(ws, ws_bytes, need)) return Q4GSW_E_WORKSPACE;
    const Range qr = range_of(q, rows_extent(s->tokens, q_ld, row, es));
    const Range orr = range_of(out, (uint64_t)s->tokens * row * es), sr = range_of(ws, need);
    if (overlap(orr, qr) || overlap(orr, cr) || overlap(sr, orr) || overlap(sr, qr) || overlap(sr, cr) ||
        over_seqs(a.sq, orr) || over_seqs(a.sq, sr))
        return Q4GSW_E_ALIAS;
    const Range tr = range_of(parents, tree ? (uint64_t)s->tokens * 4 : 0);
    if (overlap(orr, tr) || overlap(sr, tr)) return Q4GSW_E_ALIAS;
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
    a.parents = tree ? parents : nullptr;
    hipStream_t st_ = static_cast<hipStream_t>(stream);
    hipError_t e = p.kernel == AttnPlan::kPrompt ? launch_kv_prompt(a, p.waves, st_)
                   : p.kernel == AttnPlan::kTree ? launch_kv_tree(a, p.waves, st_) : launch_kv_rows(a, p.waves, st_);
    if (e == hipSuccess && p.splits > 1) e = launch_kv_join(a, st_);
    return hip_status(e);
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
        overlap(cr, range_of(v, rows_extent(sv.tokens, v_ld, row, es))) || over_seqs(sv, cr))
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
    if (overlap(kr, vr) || overlap(kr, cr) || overlap(vr, cr) || over_seqs(sv, kr) || over_seqs(sv, vr)) return Q4GSW_E_ALIAS;
    return hip_status(launch_kv_read(cv, sv, k, v, static_cast<hipStream_t>(stream)));
}

q4gsw_status q4gsw_kv_attention_workspace_bytes(const q4gsw_kv_cache* c, int32_t batch, int64_t tokens, int32_t hq,
                                                int32_t max_new, int32_t max_ctx, uint64_t* bytes) {
    if (!bytes) return Q4GSW_E_NULL;
    q4gsw_status st = check_cache_shape(c);
    if (st != Q4GSW_OK) return st;
    if ((st = check_attention(c, batch, tokens, hq, max_new, max_ctx)) != Q4GSW_OK) return st;
    // the window and the type may change the plan; the splits of either kernel grow with the span of keys
    const AttnSize n = attention_size(c->heads, c->dim, batch, hq, max_new, max_ctx, 0, kBF16);
    AttnPlan most = plan_rows(n);
    for (int i = 0; i < 4 && n.rows > kFewRows; ++i) {
        const int64_t splits = prompt_splits(n, i & 1 ? 8 : 4, i & 2);
        if (splits > most.splits) most.splits = (int)splits;
    }
    *bytes = plan_workspace(most, tokens, hq, c->dim);
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
    if ((st = read_kernel(opts, c, hq, max_new, false, &kernel)) != Q4GSW_OK) return st;
    const AttnPlan p = plan_attention(attention_size(c->heads, c->dim, batch, hq, max_new, max_ctx, window, dtype), kernel);
    *info = q4gsw_kv_plan_info{p.kernel == AttnPlan::kPrompt ? Q4GSW_KV_MANY_ROWS : Q4GSW_KV_FEW_ROWS, p.waves, p.splits};
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
    return attend(c, s, nullptr, false, q, q_ld, dtype, hq, max_new, max_ctx, window, softcap, out, ws, ws_bytes, opts, stream);
}

q4gsw_status q4gsw_kv_tree_attention_workspace_bytes(const q4gsw_kv_cache* c, int32_t batch, int64_t tokens, int32_t hq,
                                                     int32_t max_new, int32_t max_ctx, uint64_t* bytes) {
    if (max_new > kTreeMax) return bytes ? Q4GSW_E_SHAPE : Q4GSW_E_NULL;
    return q4gsw_kv_attention_workspace_bytes(c, batch, tokens, hq, max_new, max_ctx, bytes);
}

q4gsw_status q4gsw_kv_tree_attention(const q4gsw_kv_cache* c, const q4gsw_kv_seqs* s, const int32_t* parents, const void* q,
                                     int64_t q_ld, int32_t dtype, int32_t hq, int32_t max_new, int32_t max_ctx, int32_t window,
                                     float softcap, void* out, void* ws, uint64_t ws_bytes, void* stream) {
    return attend(c, s, parents, true, q, q_ld, dtype, hq, max_new, max_ctx, window, softcap, out, ws, ws_bytes, nullptr, stream);
}

q4gsw_status q4gsw_kv_tree_attention_ex(const q4gsw_kv_cache* c, const q4gsw_kv_seqs* s, const int32_t* parents,
                                        const void* q, int64_t q_ld, int32_t dtype, int32_t hq, int32_t max_new,
                                        int32_t max_ctx, int32_t window, float softcap, void* out, void* ws,
                                        uint64_t ws_bytes, const q4gsw_kv_options* opts, void* stream) {
    return attend(c, s, parents, true, q, q_ld, dtype, hq, max_new, max_ctx, window, softcap, out, ws, ws_bytes, opts, stream);
}

q4gsw_status q4gsw_kv_keep(const q4gsw_kv_cache* caches, int32_t count, const q4gsw_kv_seqs* s, const int32_t* parents,
                           const int32_t* leaf, int32_t max_new, int32_t* kept, int32_t* path, void* stream) {
    if (!caches) return Q4GSW_E_NULL;
    if (count < 1 || count > kKeepCaches) return Q4GSW_E_SHAPE;
    KvSeqs sv;
    KvView cv[kKeepCaches];
    Range cr[kKeepCaches];
    for (int i = 0; i < count; ++i) {
        const q4gsw_status st = check_cache(caches + i, cv + i, cr + i);
        if (st != Q4GSW_OK) return st;
        if (cv[i].pages != cv[0].pages || cv[i].page_size != cv[0].page_size || cv[i].heads != cv[0].heads ||
            cv[i].dim != cv[0].dim)
            return Q4GSW_E_SHAPE;
    }
    const q4gsw_status st = check_seqs(s, &sv);
    if (st != Q4GSW_OK) return st;
    if (max_new < 1 || max_new > kTreeMax || (int64_t)sv.batch * cv[0].heads > kMaxThreads / 256) return Q4GSW_E_SHAPE;
    if (!leaf || !kept || (sv.tokens > 0 && !parents)) return Q4GSW_E_NULL;
    const Range kr = range_of(kept, (uint64_t)sv.batch * 4), pr = range_of(path, path ? (uint64_t)sv.batch * max_new * 4 : 0);
    const Range ins[2] = {range_of(parents, (uint64_t)sv.tokens * 4), range_of(leaf, (uint64_t)sv.batch * 4)};
    if (overlap(kr, pr) || over_seqs(sv, kr) || over_seqs(sv, pr)) return Q4GSW_E_ALIAS;
    for (const Range& in : ins)
        if (overlap(in, kr) || overlap(in, pr)) return Q4GSW_E_ALIAS;
    for (int i = 0; i < count; ++i) {
        if (over_seqs(sv, cr[i]) || overlap(cr[i], kr) || overlap(cr[i], pr) || overlap(cr[i], ins[0]) || overlap(cr[i], ins[1]))
            return Q4GSW_E_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(cr[i], cr[j])) return Q4GSW_E_ALIAS;
    }
    return hip_status(launch_kv_keep(cv, count, sv, parents, leaf, max_new, kept, path, static_cast<hipStream_t>(stream)));
}

q4gsw_status q4gsw_logits_adjust(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                                 const q4gsw_logits_rules* r, void* out, int64_t out_ld, void* stream) {
    if (!r) return Q4GSW_E_NULL;
    if (rows < 0 || rows > kMaxM || vocab < 1 || vocab > kMaxDim || ld < vocab || out_ld < vocab || ld > kMaxDim || out_ld > kMaxDim)
        return Q4GSW_E_SHAPE;
    if (!act_dtype_ok(dtype)) return Q4GSW_E_DTYPE;
    if (r->batch < 1 || r->batch > (1 << 20)) return rows == 0 && r->batch == 0 ? Q4GSW_OK : Q4GSW_E_SHAPE;
    if (!r->cu && r->batch != rows) return Q4GSW_E_SHAPE;
    if (r->max_new < 1 || r->max_new > (r->cu && r->ids ? kTreeMax : kMaxM)) return Q4GSW_E_SHAPE;
    if (r->parents && (!r->cu || !r->ids)) return Q4GSW_E_NULL;
    if (r->history && (r->history_cols < 0 || r->history_cols > kLogitsHistory || r->history_ld < r->history_cols ||
                       r->history_ld > kMaxDim))
        return Q4GSW_E_SHAPE;
    if (r->history && !r->history_len) return Q4GSW_E_NULL;
    if (r->bias_ids && (r->bias_cols < 0 || r->bias_ld < r->bias_cols || r->bias_ld > kMaxDim)) return Q4GSW_E_SHAPE;
    if (r->bias_ids && !r->bias) return Q4GSW_E_NULL;
    if (r->mask && (r->mask_ld < (vocab + 31) / 32 || r->mask_ld > kMaxDim)) return Q4GSW_E_SHAPE;
    if (rows == 0) return Q4GSW_OK;
    if (!logits || !out) return Q4GSW_E_NULL;
    LogitsArgs a{logits, out, rows, vocab, ld, out_ld, r->batch, r->max_new, r->cu, r->history, r->history_ld, r->history_cols,
                 r->history_len, r->prompt_len, r->ids, r->parents, r->repetition, r->presence, r->frequency, r->bias_ids,
                 r->bias, r->bias_ld, r->bias_cols, r->mask, r->mask_ld, 0, 0};
    if (!r->history) a.prompt_len = nullptr;
    if (!r->cu) a.max_new = 1;
    if (!logits_launch_ok(a)) return Q4GSW_E_SHAPE;
    const int es = esize(dtype);
    const uint64_t B = (uint64_t)r->batch;
    const Range outr = range_of(out, rows_extent(rows, out_ld, vocab, es));
    auto hit = [&](const void* p, uint64_t bytes) { return p && overlap(outr, range_of(p, bytes)); };
    if (!(out == logits && out_ld == ld) && hit(logits, rows_extent(rows, ld, vocab, es))) return Q4GSW_E_ALIAS;
    if (hit(r->cu, (B + 1) * 4) || hit(r->history, rows_extent(r->batch, r->history_ld, r->history_cols, 4)) ||
        hit(r->history_len, B * 4) || hit(r->prompt_len, B * 4) || hit(r->ids, rows * 4) || hit(r->parents, rows * 4) ||
        hit(r->repetition, B * 4) || hit(r->presence, B * 4) || hit(r->frequency, B * 4) ||
        hit(r->bias_ids, rows_extent(r->batch, r->bias_ld, r->bias_cols, 4)) ||
        hit(r->bias, rows_extent(r->batch, r->bias_ld, r->bias_cols, 4)) || hit(r->mask, rows_extent(rows, r->mask_ld, (vocab + 31) / 32, 4)))
        return Q4GSW_E_ALIAS;
    return hip_status(launch_logits(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
