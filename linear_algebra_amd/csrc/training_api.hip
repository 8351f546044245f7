// Host side of the operators that train an encoder layer (attention, kept
// inputs): argument validation, work planning and launch sequences.  Layer
// descriptors travel by value with the launches; no device memory is
// allocated and nothing here can throw.
#include <algorithm>
#include <cmath>

#include "../../include/kfac.h"
#include "training.h"

namespace kfac {
namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxGrid = 0x7fffffff;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
kfac_status_t hip_status(hipError_t e) { return e == hipSuccess ? KFAC_OK : KFAC_ERR_HIP; }
bool known_dtype(kfac_dtype_t t) { return t == KFAC_F32 || t == KFAC_BF16; }

kfac_status_t enough_space(const void* ws, size_t have, size_t need) {
    return need > 0 && (ws == nullptr || !aligned(ws, kAlign) || have < need) ? KFAC_ERR_WORKSPACE : KFAC_OK;
}

struct Carver {
    uint8_t* base;
    size_t used = 0;
    explicit Carver(void* b) : base(static_cast<uint8_t*>(b)) {}
    void* take(size_t bytes) {
        void* p = base ? base + used : nullptr;
        used = align_up(used + bytes, kAlign);
        return p;
    }
};

// -------------------------------------------------------------- attention --

int buckets_of(const kfac_attention_t* f) { return (f->n_borders + 1) * (f->two_sided ? 2 : 1); }

bool attention_form(const kfac_attention_t* f) {
    if (f == nullptr) return false;
    if (f->batch < 0 || f->len_q < 0 || f->len_k < 0 || f->len_q > KFAC_MAX_LENGTH || f->len_k > KFAC_MAX_LENGTH)
        return false;
    if (f->heads < 1 || f->kv_heads < 1 || f->heads % f->kv_heads != 0 || f->heads > KFAC_MAX_DIM) return false;
    if (f->dim < 8 || f->dim > kAttnMaxDim || f->dim % 8 != 0) return false;
    if (!(f->scale > 0.0f) || !std::isfinite(f->scale)) return false;
    if (!aligned(f->lens, 4) || !aligned(f->bias, 4)) return false;
    if (f->batch > kMaxGrid / f->heads / (ceil_div(std::max<int64_t>({f->len_q, f->len_k, 1}), kAttnRows) * 8))
        return false;
    if (f->bias != nullptr) {
        if (f->n_borders < 0 || f->n_borders >= kAttnMaxBuckets || buckets_of(f) > kAttnMaxBuckets) return false;
        if (f->n_borders > 0 && f->borders == nullptr) return false;
        for (int k = 0; k < f->n_borders; ++k)
            if (f->borders[k] <= (k ? f->borders[k - 1] : 0) || f->borders[k] > (1 << 29)) return false;
    }
    return true;
}

// A tensor of `len` rows per sequence: 16-byte rows, and the rows of one tile
// within the 31 bits of a buffer offset.
bool attention_tensor(const kfac_attention_t* f, const kfac_tensor4_t* t, int64_t len, int64_t heads, int es) {
    if (t == nullptr) return false;
    if (f->batch == 0 || len == 0) return true;
    if (t->data == nullptr || !aligned(t->data, 16)) return false;
    const int64_t unit = 16 / es;
    if (f->batch > 1 && (t->stride_batch < 0 || t->stride_batch % unit != 0)) return false;
    if (heads > 1 && (t->stride_head < 0 || t->stride_head % unit != 0)) return false;
    if (len > 1 && (t->stride_row < 0 || t->stride_row % unit != 0 ||
                    t->stride_row > (int64_t(1) << 30) / (es * kAttnRows)))
        return false;
    return true;
}

int64_t lq_pad_of(const kfac_attention_t* f) { return (int64_t)align_up((size_t)f->len_q, kAttnRows); }
int64_t rel_ld_of(const kfac_attention_t* f) { return lq_pad_of(f) + 2 * kAttnRows + (int64_t)align_up((size_t)f->len_k, kAttnRows); }

// The key tiles of the pass by keys are shared out over the query heads of
// their group and over chunks of queries when there are too few of them: over
// the heads below kAttnItems (two per compute unit), and over chunks of at
// least kAttnMinChunk queries (float32 fewer: a step takes it longer) until
// every unit has a workgroup (two of them for causal rows, which differ in
// length).  A share costs its float32 rows once more in each direction.  The
// whole backward pass in bfloat16, 16 heads of 128 over 4 of keys, causal:
// 8192 rows 1838 us unshared, 1030 shared; 2048 rows 474 unshared, 211 with
// one workgroup per unit, 187 with two.  Not causal, 2 sequences of 512, 16
// heads of 64: 46 unshared, 49 with one per unit, 54 with two.  Chunks of at
// least 64 queries instead: 128 rows, 16 heads of 64, 24.7 us instead of 21.8,
// 512 causal rows, 16 heads of 128 over 4, 59.5 instead of 53.2; in float32,
// 214 x 61, 24 heads of 96, 62 instead of 55.
constexpr int64_t kAttnItems = 512;
constexpr int64_t kAttnUnits = 256;
constexpr int64_t kAttnMinChunk = 128, kAttnMinChunkF32 = 32;

// Passes by queries with fewer workgroups of 128 queries than this take 32
// queries per workgroup and share out the keys over its waves.  Forward in
// bfloat16, 16 heads of 64, in us as they are / shared out: 1 sequence of 512
// (64 workgroups) 15.4 / 11.4, 2 (128) 16.0 / 13.5, 3 (192) 16.7 / 18.9, 4
// (256) 17.3 / 22.0; one row of 8192 keys 151 / 76.  float32, 333 queries of
// 401 keys, 18 heads of 72 (54): 54 / 26.
constexpr int64_t kAttnDeep = 192;

struct AttnShares {
    int32_t parts = 1, qchunk = 1;
};

AttnShares shares_of(const kfac_attention_t* f, bool bf16, int64_t ktiles, int64_t step) {
    AttnShares s;
    const int64_t qt = std::max<int64_t>(1, ceil_div(f->len_q, step)), group = f->heads / f->kv_heads;
    const int64_t tiles = f->batch * f->kv_heads * ktiles;
    s.qchunk = (int32_t)qt;
    if (tiles == 0 || tiles >= kAttnItems) return s;
    const int64_t fill = (f->causal ? 2 : 1) * kAttnUnits / (tiles * group);
    const int64_t most = qt * step / (bf16 ? kAttnMinChunk : kAttnMinChunkF32);
    const int64_t chunks = std::max<int64_t>(1, std::min(fill, most));
    s.qchunk = (int32_t)ceil_div(qt, chunks);
    s.parts = (int32_t)(group * ceil_div(qt, s.qchunk));
    return s;
}

// Fills the sizes and plan of a call and carves its workspace; returns the bytes needed.
size_t attention_args(const kfac_attention_t* f, kfac_dtype_t dtype, bool backward, void* ws, AttnArgs& a) {
    a.lens = f->lens;
    a.batch = (int32_t)f->batch;
    a.len_q = (int32_t)f->len_q;
    a.len_k = (int32_t)f->len_k;
    a.heads = f->heads;
    a.kv_heads = f->kv_heads;
    a.group = f->heads / f->kv_heads;
    a.dim = f->dim;
    a.lq_pad = (int32_t)lq_pad_of(f);
    a.rel_ld = rel_ld_of(f);
    a.deep = f->batch * f->heads * ceil_div(f->len_q, kAttnRows) < kAttnDeep;
    a.qtiles = (int32_t)ceil_div(f->len_q, a.deep ? 32 : kAttnRows);
    a.causal = f->causal != 0;
    a.scale = f->scale;
    a.scale2 = (float)((double)f->scale * 1.4426950408889634);
    Carver c(ws);
    if (f->bias != nullptr) {
        // offsets (key - query position) from far_hi up, and from far_lo down, lie in one bucket each
        const int last = f->n_borders ? f->borders[f->n_borders - 1] : 0;
        a.bias = f->bias;
        a.buckets = buckets_of(f);
        a.far_lo = -last;
        a.far_lo_bucket = f->n_borders;
        a.far_hi = f->two_sided ? std::max(last, 1) : 0;
        a.far_hi_bucket = f->two_sided ? 2 * f->n_borders + 1 : 0;
        a.borders.n = f->n_borders;
        a.borders.two_sided = f->two_sided != 0;
        std::fill_n(std::copy_n(f->borders, f->n_borders, a.borders.at), kAttnMaxBuckets - f->n_borders, INT32_MAX);
        const int64_t near = (int64_t)a.far_hi - a.far_lo + 1 + 2 * kAttnPad;
        if (near <= kAttnNear) a.near_n = (int32_t)near;
        else a.rel = static_cast<float*>(c.take(sizeof(float) * (size_t)(f->heads * a.rel_ld)));
    }
    if (backward) {
        const bool bf16 = dtype == KFAC_BF16;
        a.ktiles = (int32_t)ceil_div(f->len_k, kAttnRows);
        const AttnShares s = shares_of(f, bf16, a.ktiles, attn_step_queries(bf16, f->dim));
        a.parts = s.parts;
        a.qchunk = s.qchunk;
        const size_t rows = (size_t)(f->batch * f->heads * a.lq_pad);
        a.stats = static_cast<float*>(c.take(sizeof(float) * 2 * rows));
        if (f->bias != nullptr)
            a.part = static_cast<float*>(
                c.take(sizeof(float) * (size_t)(f->batch * f->heads * a.qtiles * 4) * (size_t)a.buckets));
        if (a.parts > 1)
            a.kv_part = static_cast<float*>(
                c.take(sizeof(float) * 2 * (size_t)a.parts * (size_t)(f->batch * f->kv_heads * f->len_k) * f->dim));
    }
    return c.used;
}

AttnTensor tensor_of(const kfac_tensor4_t* t) { return AttnTensor{t->data, t->stride_batch, t->stride_row, t->stride_head}; }

// ------------------------------------------------------------ checkpoints --

bool keep_shape(int64_t rows, int64_t d) { return rows >= 1 && rows <= 0x7fffffff && d >= 1 && d <= KFAC_MAX_DIM; }
bool keep_pointers(const uint8_t* codes, const uint8_t* scales) {
    return codes != nullptr && scales != nullptr && aligned(codes, 16);
}

// Store and load: layers in groups that travel with one launch each.
template <typename F>
kfac_status_t keep_run(bool load, int n, const void* const* x, const int64_t* rows, const int64_t* cols, const int64_t* da,
                       kfac_dtype_t dtype, uint8_t* const* codes, uint8_t* const* scales, hipStream_t stream, F launch) {
    const bool bf16 = dtype == KFAC_BF16;
    for (int first = 0; first < n; first += kKeepGroup) {
        KeepLaunch l{};
        int64_t blocks = 0;
        l.n = std::min(kKeepGroup, n - first);
        for (int k = 0; k < l.n; ++k) {
            const int i = first + k;
            KeepLayer& y = l.layer[k];
            y.x = const_cast<void*>(x[i]);
            y.codes = codes[i];
            y.scales = scales[i];
            y.rows = rows[i];
            y.cols = (int32_t)cols[i];
            y.da = (int32_t)da[i];
            y.groups = (int32_t)ceil_div(load ? cols[i] : da[i], kKeepThreads * (bf16 ? 2 : 1));
            y.block_begin = blocks;
            blocks += ceil_div(rows[i], load ? kKeepBlock / 2 : kKeepBlock) * y.groups;
        }
        if (blocks > kMaxGrid) return KFAC_ERR_UNSUPPORTED;
        const hipError_t e = launch(l, blocks, bf16, stream);
        if (e != hipSuccess) return KFAC_ERR_HIP;
    }
    return KFAC_OK;
}

// Tiles go to the compute units in rounds of kKeepRound.  The tiles of the
// last, incomplete round are split along the rows into chunks of at least
// kKeepMinChunk blocks, for the number of rounds that costs least: a round
// takes its chunk's blocks and about kKeepBegin more, and the partial tiles of
// a full round, written once and read once, take as long as kKeepJoin blocks.
// 4096 rows, in us without a split / with the fewest chunks that fill one
// round / two rounds: factor of width 1025 (45 tiles) 43 / 25.5 / 29, of width
// 2049 (153 tiles) 48 / 48 / 38, gradient 1024 x 1025 (72 tiles) 39 / 27 / 33;
// split in full, the 33 x 8 tiles of a 1024 x 4097 gradient take 75 instead
// of 54.  Chunks of 2 blocks: 128 rows, 1024 x 2049 in float32, 30 instead of
// 12.5.
constexpr int64_t kKeepRound = 256;
constexpr int64_t kKeepMinChunk = 8;
constexpr int64_t kKeepBegin = 4;
constexpr int64_t kKeepJoin = 12;

int64_t split_of(int64_t tiles, int64_t blocks) {
    int64_t best = 1, least = INT64_MAX;
    for (int64_t round = 0; tiles > 0 && round <= 4; ++round) {
        // as many chunks as fit this many rounds
        const int64_t s = std::max<int64_t>(1, std::min(round * kKeepRound / tiles, blocks / kKeepMinChunk));
        const int64_t cost = ceil_div(tiles * s, kKeepRound) * (ceil_div(blocks, s) + kKeepBegin) +
                             (s > 1 ? kKeepJoin * tiles * s / kKeepRound : 0);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

struct KeepPlan {
    int64_t items = 0, red = 0, cut = 0;
    size_t part_bytes = 0;
};

KeepPlan plan_products(KeepProb* p, int n, bool factor) {
    KeepPlan plan;
    int64_t tiles = 0, longest = 0;
    for (int k = 0; k < n; ++k) {
        p[k].tiles_m = (int32_t)ceil_div(p[k].m, kKeepTile);
        p[k].tiles_n = (int32_t)ceil_div(p[k].da, kKeepTile);
        p[k].ntiles = factor ? p[k].tiles_n * (p[k].tiles_n + 1) / 2 : p[k].tiles_m * p[k].tiles_n;
        p[k].blocks = (int32_t)ceil_div(p[k].rows, kKeepBlock);
        tiles += p[k].ntiles;
        longest = std::max<int64_t>(longest, p[k].blocks);
    }
    // the last round's tiles are the last tiles of the last problems
    int64_t whole = tiles / kKeepRound * kKeepRound;
    plan.cut = whole;
    const int64_t want = split_of(tiles - whole, longest);
    for (int k = 0; k < n; ++k) {
        const int64_t split = std::max<int64_t>(1, std::min<int64_t>(want, p[k].blocks / kKeepMinChunk));
        p[k].kchunk = (int32_t)align_up((size_t)ceil_div(p[k].blocks, split), 2);
        p[k].ksplit = (int32_t)ceil_div(p[k].blocks, p[k].kchunk);
        p[k].whole = p[k].ksplit == 1 ? p[k].ntiles : (int32_t)std::min<int64_t>(whole, p[k].ntiles);
        whole -= std::min<int64_t>(whole, p[k].ntiles);
        const int64_t rest = p[k].ntiles - p[k].whole;
        p[k].item_begin = plan.items;
        p[k].red_begin = plan.red;
        plan.items += p[k].whole + rest * p[k].ksplit;
        plan.red += rest;
        plan.part_bytes += sizeof(float) * (size_t)(rest * p[k].ksplit) * kKeepTile * kKeepTile;
    }
    return plan;
}

// Partial tiles of a group of layers; groups run one after another on the
// stream and share the space.
size_t products_ws(int n, const int64_t* rows, const int64_t* m, const int64_t* da, bool factor) {
    size_t most = 0;
    for (int first = 0; first < n; first += kKeepGroup) {
        KeepProb p[kKeepGroup] = {};
        const int c = std::min(kKeepGroup, n - first);
        for (int k = 0; k < c; ++k) {
            p[k].rows = rows[first + k];
            p[k].m = (int32_t)m[first + k];
            p[k].da = (int32_t)da[first + k];
        }
        most = std::max(most, plan_products(p, c, factor).part_bytes);
    }
    return most;
}

bool products_shape(int n, const int64_t* rows, const int64_t* m, const int64_t* da) {
    if (n < 1 || n > KFAC_MAX_COUNT || rows == nullptr || m == nullptr || da == nullptr) return false;
    for (int i = 0; i < n; ++i)
        if (!keep_shape(rows[i], da[i]) || m[i] < 1 || m[i] > KFAC_MAX_DIM) return false;
    return true;
}

kfac_status_t products_run(int n, const void* const* g, const uint8_t* const* codes, const uint8_t* const* scales,
                           const int64_t* rows, const int64_t* m, const int64_t* da, kfac_dtype_t dtype, float* const* out,
                           float eps, int first_step, void* workspace, hipStream_t stream) {
    const bool factor = g == nullptr, bf16 = dtype == KFAC_BF16;
    for (int first = 0; first < n; first += kKeepGroup) {
        KeepProbs l{};
        l.n = std::min(kKeepGroup, n - first);
        l.eps = eps;
        l.first_step = first_step;
        bool words = true;
        for (int k = 0; k < l.n; ++k) {
            const int i = first + k;
            KeepProb& p = l.p[k];
            p.codes = codes[i];
            p.scales = scales[i];
            p.out = out[i];
            p.rows = rows[i];
            p.m = (int32_t)m[i];
            p.da = (int32_t)da[i];
            p.alpha = (float)(1.0 / (double)rows[i]);
            if (!factor) {
                p.g = g[i];
                words = words && aligned(g[i], 4) && (!bf16 || m[i] % 2 == 0);
            }
        }
        const KeepPlan plan = plan_products(l.p, l.n, factor);
        if (plan.items > kMaxGrid || 16 * plan.red > kMaxGrid) return KFAC_ERR_UNSUPPORTED;
        l.cut = (int32_t)plan.cut;
        float* part = static_cast<float*>(workspace);
        for (int k = 0; k < l.n; ++k) {
            l.p[k].part = part;
            part += (size_t)(l.p[k].ntiles - l.p[k].whole) * l.p[k].ksplit * kKeepTile * kKeepTile;
        }
        hipError_t e = factor ? launch_keep_factor(l, plan.items, stream) : launch_keep_grad(l, plan.items, bf16, words, stream);
        if (e == hipSuccess) e = launch_keep_reduce(l, plan.red, factor, stream);
        if (e != hipSuccess) return KFAC_ERR_HIP;
    }
    return KFAC_OK;
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" {

// -------------------------------------------------------------- attention --

size_t kfac_attention_workspace_size(const kfac_attention_t* form, kfac_dtype_t dtype, int backward) {
    if (!attention_form(form) || !known_dtype(dtype)) return SIZE_MAX;
    AttnArgs a{};
    return attention_args(form, dtype, backward != 0, nullptr, a);
}

kfac_status_t kfac_attention_forward(const kfac_attention_t* form, kfac_dtype_t dtype, const kfac_tensor4_t* q,
                                     const kfac_tensor4_t* k, const kfac_tensor4_t* v, const kfac_tensor4_t* out,
                                     float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!attention_form(form) || !known_dtype(dtype)) return KFAC_ERR_INVALID_VALUE;
    const int es = dtype == KFAC_BF16 ? 2 : 4;
    if (!attention_tensor(form, q, form->len_q, form->heads, es) ||
        !attention_tensor(form, out, form->len_q, form->heads, es) ||
        !attention_tensor(form, k, form->len_k, form->kv_heads, es) ||
        !attention_tensor(form, v, form->len_k, form->kv_heads, es))
        return KFAC_ERR_INVALID_VALUE;
    const bool none = form->batch == 0 || form->len_q == 0;
    if (!none && (lse == nullptr || !aligned(lse, 4))) return KFAC_ERR_INVALID_VALUE;
    AttnArgs a{};
    const size_t need = attention_args(form, dtype, false, workspace, a);
    const kfac_status_t space = enough_space(workspace, workspace_bytes, need);
    if (space != KFAC_OK) return space;
    if (none) return KFAC_OK;
    a.q = tensor_of(q);
    a.k = tensor_of(k);
    a.v = tensor_of(v);
    a.out = tensor_of(out);
    a.lse = lse;
    hipError_t e = a.rel != nullptr ? launch_attn_bias(a, stream) : hipSuccess;
    if (e == hipSuccess) e = launch_attn_forward(a, dtype == KFAC_BF16, stream);
    return hip_status(e);
}

kfac_status_t kfac_attention_backward(const kfac_attention_t* form, kfac_dtype_t dtype, const kfac_tensor4_t* q,
                                      const kfac_tensor4_t* k, const kfac_tensor4_t* v, const kfac_tensor4_t* out,
                                      const float* lse, const kfac_tensor4_t* dout, const kfac_tensor4_t* dq,
                                      const kfac_tensor4_t* dk, const kfac_tensor4_t* dv, float* dbias, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
    if (!attention_form(form) || !known_dtype(dtype)) return KFAC_ERR_INVALID_VALUE;
    const int es = dtype == KFAC_BF16 ? 2 : 4;
    for (const kfac_tensor4_t* t : {q, out, dout, dq})
        if (!attention_tensor(form, t, form->len_q, form->heads, es)) return KFAC_ERR_INVALID_VALUE;
    for (const kfac_tensor4_t* t : {k, v, dk, dv})
        if (!attention_tensor(form, t, form->len_k, form->kv_heads, es)) return KFAC_ERR_INVALID_VALUE;
    const bool no_rows = form->batch == 0 || form->len_q == 0;
    if (!no_rows && (lse == nullptr || !aligned(lse, 4))) return KFAC_ERR_INVALID_VALUE;
    if ((form->bias != nullptr) != (dbias != nullptr) || !aligned(dbias, 4)) return KFAC_ERR_INVALID_VALUE;
    AttnArgs a{};
    const size_t need = attention_args(form, dtype, true, workspace, a);
    const kfac_status_t space = enough_space(workspace, workspace_bytes, need);
    if (space != KFAC_OK) return space;
    a.q = tensor_of(q);
    a.k = tensor_of(k);
    a.v = tensor_of(v);
    a.out = tensor_of(out);
    a.dout = tensor_of(dout);
    a.dq = tensor_of(dq);
    a.dk = tensor_of(dk);
    a.dv = tensor_of(dv);
    a.lse = const_cast<float*>(lse);
    a.dbias = dbias;
    const bool bf16 = dtype == KFAC_BF16;
    hipError_t e = a.rel != nullptr && !no_rows ? launch_attn_bias(a, stream) : hipSuccess;
    if (e == hipSuccess && !no_rows) e = launch_attn_dq(a, bf16, stream);
    if (e == hipSuccess) e = launch_attn_dkdv(a, bf16, stream);
    if (e == hipSuccess && a.parts > 1) e = launch_attn_kv_sum(a, bf16, stream);
    return hip_status(e);
}

// ------------------------------------------------------------ checkpoints --

kfac_status_t kfac_checkpoint_store(int n, const void* const* x, const int64_t* rows, const int64_t* d, int ones,
                                    kfac_dtype_t dtype, uint8_t* const* codes, uint8_t* const* scales,
                                    hipStream_t stream) {
    if (n < 1 || n > KFAC_MAX_COUNT || !x || !rows || !d || !codes || !scales || !known_dtype(dtype) ||
        (ones != 0 && ones != 1))
        return KFAC_ERR_INVALID_VALUE;
    for (int i = 0; i < n; ++i)
        if (!keep_shape(rows[i], d[i]) || d[i] + ones > KFAC_MAX_DIM || x[i] == nullptr ||
            !aligned(x[i], dtype == KFAC_BF16 ? 2 : 4) || !keep_pointers(codes[i], scales[i]))
            return KFAC_ERR_INVALID_VALUE;
    for (int first = 0; first < n; first += kKeepGroup) {
        const int c = std::min(kKeepGroup, n - first);
        int64_t da[kKeepGroup];
        for (int k = 0; k < c; ++k) da[k] = d[first + k] + ones;
        const kfac_status_t st =
            keep_run(false, c, x + first, rows + first, d + first, da, dtype, codes + first, scales + first, stream,
                     launch_keep_store);
        if (st != KFAC_OK) return st;
    }
    return KFAC_OK;
}

kfac_status_t kfac_checkpoint_load(int n, const uint8_t* const* codes, const uint8_t* const* scales, const int64_t* rows,
                                   const int64_t* d, const int64_t* cols, kfac_dtype_t dtype, void* const* y,
                                   hipStream_t stream) {
    if (n < 1 || n > KFAC_MAX_COUNT || !y || !rows || !d || !cols || !codes || !scales || !known_dtype(dtype))
        return KFAC_ERR_INVALID_VALUE;
    for (int i = 0; i < n; ++i)
        if (!keep_shape(rows[i], d[i]) || cols[i] < 1 || cols[i] > d[i] || y[i] == nullptr ||
            !aligned(y[i], dtype == KFAC_BF16 ? 2 : 4) || !keep_pointers(codes[i], scales[i]))
            return KFAC_ERR_INVALID_VALUE;
    return keep_run(true, n, y, rows, cols, d, dtype, const_cast<uint8_t* const*>(codes), const_cast<uint8_t* const*>(scales),
                    stream, launch_keep_load);
}

size_t kfac_checkpoint_factors_workspace_size(int n, const int64_t* rows, const int64_t* d) {
    return products_shape(n, rows, d, d) ? products_ws(n, rows, d, d, true) : SIZE_MAX;
}

kfac_status_t kfac_checkpoint_factors(int n, const uint8_t* const* codes, const uint8_t* const* scales,
                                      const int64_t* rows, const int64_t* d, float* const* m, float eps, int first_step,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!products_shape(n, rows, d, d) || !codes || !scales || !m) return KFAC_ERR_INVALID_VALUE;
    if (!(eps >= 0.0f && eps <= 1.0f)) return KFAC_ERR_INVALID_VALUE;
    for (int i = 0; i < n; ++i)
        if (!keep_pointers(codes[i], scales[i]) || m[i] == nullptr || !aligned(m[i], 4)) return KFAC_ERR_INVALID_VALUE;
    const kfac_status_t space = enough_space(workspace, workspace_bytes, products_ws(n, rows, d, d, true));
    if (space != KFAC_OK) return space;
    return products_run(n, nullptr, codes, scales, rows, d, d, KFAC_F32, m, eps, first_step != 0, workspace, stream);
}

size_t kfac_checkpoint_grad_workspace_size(int n, const int64_t* rows, const int64_t* d_out, const int64_t* d) {
    return products_shape(n, rows, d_out, d) ? products_ws(n, rows, d_out, d, false) : SIZE_MAX;
}

kfac_status_t kfac_checkpoint_grad(int n, const void* const* g, const uint8_t* const* codes,
                                   const uint8_t* const* scales, const int64_t* rows, const int64_t* d_out,
                                   const int64_t* d, kfac_dtype_t dtype, float* const* mat, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
    if (!products_shape(n, rows, d_out, d) || !g || !codes || !scales || !mat || !known_dtype(dtype))
        return KFAC_ERR_INVALID_VALUE;
    for (int i = 0; i < n; ++i)
        if (!keep_pointers(codes[i], scales[i]) || g[i] == nullptr || !aligned(g[i], dtype == KFAC_BF16 ? 2 : 4) ||
            mat[i] == nullptr || !aligned(mat[i], 4))
            return KFAC_ERR_INVALID_VALUE;
    const kfac_status_t space = enough_space(workspace, workspace_bytes, products_ws(n, rows, d_out, d, false));
    if (space != KFAC_OK) return space;
    return products_run(n, g, codes, scales, rows, d_out, d, dtype, mat, 0.0f, 1, workspace, stream);
}

}  // extern "C"
