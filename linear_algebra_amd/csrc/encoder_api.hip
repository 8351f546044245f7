// Host side of the operators around an encoder layer's products (layer norm,
// the gated feed-forward block, gradient norm and clipping): argument validation, work planning and launch
// sequences.  Tables travel by value with the launches; no device memory is
// allocated and nothing here can throw.
#include <algorithm>
#include <cmath>

#include "../../include/kfac.h"
#include "encoder.h"

namespace kfac {
namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
kfac_status_t hip_status(hipError_t e) { return e == hipSuccess ? KFAC_OK : KFAC_ERR_HIP; }
bool known_dtype(kfac_dtype_t t) { return t == KFAC_F32 || t == KFAC_BF16; }
size_t size_of(kfac_dtype_t t) { return t == KFAC_BF16 ? 2 : 4; }

kfac_status_t enough_space(const void* ws, size_t have, size_t need) {
    return need > 0 && (ws == nullptr || !aligned(ws, kAlign) || have < need) ? KFAC_ERR_WORKSPACE : KFAC_OK;
}

// ------------------------------------------------------------- layer norm --

bool norm_shape(int64_t rows, int64_t d) { return rows >= 0 && rows <= INT32_MAX && d >= 1 && d <= KFAC_MAX_DIM; }

bool norm_rows(const void* p, int64_t stride, int64_t rows, int64_t d, kfac_dtype_t dtype) {
    if (rows == 0) return true;
    return p != nullptr && aligned(p, size_of(dtype)) && (rows == 1 || (stride >= d && stride <= (int64_t(1) << 40)));
}

// A vector of the weight's type; NULL where it may be left out.
bool norm_vector(const void* p, kfac_dtype_t dtype) { return aligned(p, size_of(dtype)); }

bool norm_types(kfac_dtype_t dtype, kfac_dtype_t weight_dtype) {
    return known_dtype(dtype) && (weight_dtype == KFAC_F32 || weight_dtype == dtype);
}

// (of the type that needs more)
size_t norm_ws(int64_t rows, int64_t d) { return (size_t)norm_parts(rows, d, true) * 2 * (size_t)norm_pitch(d) * sizeof(float); }

// -------------------------------------------------------- gradient norm --

struct Range {
    uintptr_t begin, end;
};

// The tensors' sizes, addresses and types; writes the number of all chunks.
bool clip_tensors(int n, const void* const* g, const int64_t* count, const kfac_dtype_t* dtype, int64_t& chunks) {
    if (n < 1 || n > KFAC_MAX_COUNT || g == nullptr || count == nullptr || dtype == nullptr) return false;
    chunks = 0;
    for (int i = 0; i < n; ++i) {
        if (!known_dtype(dtype[i]) || count[i] < 0 || count[i] > (int64_t(1) << 37)) return false;
        if (count[i] > 0 && (g[i] == nullptr || !aligned(g[i], size_of(dtype[i])))) return false;
        chunks += ceil_div(count[i], kClipChunk);
    }
    return true;
}

// No tensor may be written while another one's workgroups read it: whatever
// is written, the norm included, lies apart from everything but the gradient
// it stands for.
bool clip_apart(int n, const void* const* g, void* const* out, const int64_t* count, const kfac_dtype_t* dtype,
                const float* norm) {
    Range r[2 * KFAC_MAX_COUNT];
    int m = 0;
    bool sorted = true, apart = true;
    const uintptr_t one = reinterpret_cast<uintptr_t>(norm);
    auto take = [&](const void* p, size_t bytes) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        apart = apart && (one + sizeof(float) <= at || at + bytes <= one);
        r[m++] = {at, at + bytes};
        sorted = sorted && (m < 2 || r[m - 2].begin <= at);
    };
    for (int i = 0; i < n; ++i)
        if (count[i] > 0) take(g[i], (size_t)count[i] * size_of(dtype[i]));
    for (int i = 0; i < n; ++i)
        if (count[i] > 0 && out[i] != g[i]) take(out[i], (size_t)count[i] * size_of(dtype[i]));
    if (!sorted) std::sort(r, r + m, [](const Range& a, const Range& b) { return a.begin < b.begin; });
    for (int k = 1; k < m; ++k)
        if (r[k].begin < r[k - 1].end) return false;
    return apart;
}

int clip_parts(int64_t chunks, int64_t all) {
    return (int)std::max<int64_t>(1, std::min(chunks, kClipBlocks * chunks / std::max<int64_t>(all, 1)));
}

// The table of the tensors from `first` on; returns the next table's first.
int clip_table(int first, int n, const void* const* g, void* const* out, const int64_t* count, const kfac_dtype_t* dtype,
               ClipTable& t) {
    t.n = 0;
    t.chunks = 0;
    int i = first;
    for (; i < n && t.n < kClipGroup; ++i) {
        if (count[i] == 0) continue;
        const int64_t c = ceil_div(count[i], kClipChunk);
        ClipTensor& e = t.t[t.n++];
        e.g = g[i];
        e.out = out ? out[i] : nullptr;
        e.begin = t.chunks;
        e.last = (uint32_t)(count[i] - (c - 1) * kClipChunk) | (dtype[i] == KFAC_BF16 ? kClipBf16 : 0u);
        t.chunks += (uint32_t)c;
    }
    return i;
}

int clip_groups(int n) { return (n + kClipGroup - 1) / kClipGroup; }
size_t clip_ws(int n) { return (size_t)(kClipBlocks + clip_groups(n)) * sizeof(double); }

// The sums of squares of every table; t is left as the last launch's.
kfac_status_t clip_squares(int n, const void* const* g, const int64_t* count, const kfac_dtype_t* dtype, int64_t chunks,
                           float* norm, void* workspace, ClipTable& t, hipStream_t stream) {
    t.part = static_cast<double*>(workspace);
    t.norm = norm;
    t.parts = 0;
    for (int i = 0; i < n;) {
        i = clip_table(i, n, g, nullptr, count, dtype, t);
        if (t.n == 0) continue;
        t.first_part = t.parts;
        const int blocks = clip_parts(t.chunks, chunks);
        t.parts += blocks;
        if (launch_clip_squares(t, blocks, stream) != hipSuccess) return KFAC_ERR_HIP;
    }
    return KFAC_OK;
}

// ------------------------------------------------------------------ gated --

constexpr int64_t kMaxThreads = 0xffffffff;   // of a launch along one dimension

struct Carver {
    uint8_t* base;
    size_t used = 0;
    explicit Carver(void* b) : base(static_cast<uint8_t*>(b)) {}
    template <typename T>
    T* take(size_t bytes) {
        uint8_t* p = base ? base + used : nullptr;
        used = align_up(used + bytes, kAlign);
        return reinterpret_cast<T*>(p);
    }
};

bool gated_shape(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype) {
    return rows >= 0 && rows <= INT32_MAX && d >= 1 && d <= KFAC_MAX_DIM && width >= 1 && width <= KFAC_MAX_DIM &&
           known_dtype(dtype);
}

// A matrix that the products read as it is, or that is repacked first: float32
// into planes, bfloat16 of an odd width to an even pitch.
struct GatedMatrix {
    const void* src = nullptr;
    uint16_t* packed = nullptr;
    int64_t rows = 0;
    int32_t cols = 0, pitch = 0;
    bool repack = false, f32 = false;

    GatedMatrix(int64_t r, int64_t c, kfac_dtype_t dtype, Carver& ws) : rows(r), cols((int32_t)c) {
        f32 = dtype == KFAC_F32;
        repack = f32 || c % 2 != 0;
        pitch = repack ? (int32_t)align_up((size_t)c, 8) : cols;
        if (repack) packed = ws.take<uint16_t>((size_t)plane() * (f32 ? 3 : 1) * 2);
    }
    int64_t plane() const { return rows * pitch; }
    // limit: its rows where the reduction runs along them, else its columns
    ProdOperand operand(int32_t limit, int32_t apart = 0) const {
        ProdOperand o{};
        o.p = repack ? packed : static_cast<const uint16_t*>(src);
        o.plane = plane();
        o.bytes = plane() * 2;
        o.ld = pitch;
        o.limit = limit;
        o.apart = apart;
        return o;
    }
    void enter(RepackTable& t, int64_t& blocks) const {
        if (!repack || rows == 0) return;
        RepackMatrix& m = t.m[t.n++];
        m.src = src;
        m.dst = packed;
        m.rows = rows;
        m.plane = plane();
        m.cols = cols;
        m.pitch = pitch;
        m.begin = (uint32_t)blocks;
        m.bf16 = !f32;
        blocks += ceil_div(rows * (pitch / 8), 256);
    }
};

// One product's size; forward: N columns of each projection.
struct ProdSize {
    int64_t M = 0, N = 0, K = 0;
    bool forward = false;
    int64_t tiles_m(const ProdForm& f) const { return ceil_div(M, f.m); }
    int64_t tiles_n(const ProdForm& f) const { return ceil_div(N, forward ? f.n / 2 : f.n); }
    int64_t tiles(const ProdForm& f) const { return tiles_m(f) * tiles_n(f); }
    uint32_t slabs() const { return (uint32_t)std::max<int64_t>(1, ceil_div(K, 64)); }
};

// How products that share a launch run (dx and dW; the forward one alone):
// their form, and how many of each one's last tiles are shared out along the
// reduction so that the last round of the launch, too, fills the card.  The form and the length
// of a share are those of the least time by the forms' measured costs: dW of
// 25088 x 2304 x 9216 by itself, 324 tiles of 256 x 256, took 1200 us in two
// rounds, 880 with 256 whole tiles and 68 in three shares; by 128 x 128, 1126.
struct PairPlan {
    int form = 0;
    int64_t tiles[2] = {0, 0}, whole[2] = {0, 0}, splits[2] = {1, 1}, kchunk[2] = {64, 64};
    size_t part_bytes = 0;
    double time = 0.0;      // us, as the costs have it

    int64_t items() const { return whole[0] + whole[1] + (tiles[0] - whole[0]) * splits[0] + (tiles[1] - whole[1]) * splits[1]; }
    bool fits() const {
        return tiles[0] <= INT32_MAX && tiles[1] <= INT32_MAX && items() <= kMaxThreads / kProdForms[form].threads;
    }

    // the forms [from, to]
    PairPlan(const ProdSize (&size)[2], int from, int to) {
        bool any = false;
        for (int f = from; f <= to; ++f) {
            const ProdForm& pf = kProdForms[f];
            const int64_t n[2] = {size[0].tiles(pf), size[1].tiles(pf)};
            const uint32_t s[2] = {size[0].slabs(), size[1].slabs()};   // (their quotients in 32 bits: this runs on every call)
            const int64_t total = n[0] * s[0] + n[1] * s[1];
            // no less than the work shared out evenly
            if (any && (double)total / pf.slots * pf.step + pf.rest >= time) continue;
            // which product's tiles are all shared out (2: neither's): one whose
            // tiles take longer than the launch would
            for (int all = 0; all <= 2; ++all) {
                if (all < 2 && (n[all] == 0 || (int64_t)s[all] * pf.slots <= total)) continue;
                int64_t first[2] = {all == 0 ? 0 : n[0], all == 1 ? 0 : n[1]};
                const int64_t full = (first[0] + first[1]) / pf.slots * pf.slots;
                first[0] = std::min(first[0], full);
                first[1] = std::min(first[1], full - first[0]);
                const int64_t rest[2] = {n[0] - first[0], n[1] - first[1]};
                const int64_t work = rest[0] * s[0] + rest[1] * s[1];
                const uint32_t most = std::max(s[0], s[1]);
                auto shares = [&](int k, uint32_t length) { return (s[k] + length - 1) / length; };
                auto count = [&](uint32_t length) { return rest[0] * shares(0, length) + rest[1] * shares(1, length); };
                double rounds = 0.0;
                if (full > 0) {
                    const double mean = (double)(first[0] * s[0] + first[1] * s[1]) / pf.slots;
                    const uint32_t one = std::max(first[0] ? s[0] : 0, first[1] ? s[1] : 0);
                    rounds = std::max(mean, (double)one) * pf.step + (double)(full / pf.slots) * pf.rest;
                }
                // no shares; shares of the least length (256 steps at least)
                // whose number fits one or two rounds; or of the shorter
                // product's, which stays whole
                for (int turns = 0; turns <= (work > 0 ? 3 : 0); ++turns) {
                    uint32_t length = turns == 3 ? std::max<uint32_t>(4, std::min(s[0], s[1])) : most;
                    if (turns == 1 || turns == 2) {
                        uint32_t low = (uint32_t)std::min<int64_t>(most, std::max<int64_t>(4, ceil_div(work, pf.slots * turns)));
                        while (low < length) {
                            const uint32_t mid = (low + length) / 2;
                            if (count(mid) <= pf.slots * turns) length = mid;
                            else low = mid + 1;
                        }
                    }
                    uint32_t parts[2], chunk[2], longest = 0;
                    int64_t items = 0;
                    size_t bytes = 0;
                    for (int k = 0; k < 2; ++k) {
                        parts[k] = std::min(shares(k, length), 64u);
                        chunk[k] = shares(k, parts[k]);
                        parts[k] = shares(k, chunk[k]);
                        if (rest[k] == 0) continue;
                        items += rest[k] * parts[k];
                        longest = std::max(longest, chunk[k]);
                        if (parts[k] > 1) bytes += (size_t)(rest[k] * parts[k]) * (size_t)(pf.m * pf.n) * 4;
                    }
                    // the last round's time; the shares, written and read at 4.5 TB/s, and a launch
                    const double tail = std::max((double)work / pf.slots, (double)longest) * pf.step +
                                        (double)ceil_div(items, pf.slots) * pf.rest;
                    const double t = rounds + tail + (bytes ? 5.0 + 2.0 * (double)bytes / 4.5e6 : 0.0);
                    if (any && t >= time) continue;
                    any = true;
                    time = t;
                    form = f;
                    part_bytes = bytes;
                    for (int k = 0; k < 2; ++k) {
                        tiles[k] = n[k];
                        whole[k] = parts[k] > 1 ? first[k] : n[k];
                        splits[k] = parts[k];
                        kchunk[k] = (int64_t)chunk[k] * 64;
                    }
                }
            }
        }
    }
};

// The backward pass's row chunks for the elementwise part.
struct GradPlan {
    int64_t chunk, parts;
    GradPlan(int64_t rows, int64_t width, kfac_dtype_t dtype) {
        const int64_t columns = ceil_div(width, 64 * (dtype == KFAC_BF16 ? 8 : 4));
        const int64_t want = std::max<int64_t>(1, std::min(ceil_div(1024, columns), ceil_div(rows, 4)));
        chunk = (int64_t)align_up((size_t)std::max<int64_t>(1, ceil_div(rows, want)), 4);
        parts = ceil_div(rows, chunk);
    }
};

// The workspace of a call, carved (from no address: to count its bytes).
struct GatedSpace {
    Carver ws;
    GatedMatrix x, w, dpre;
    ProdSize size[2];       // dx (or the forward product), dW; empty where they are not formed
    PairPlan plan;
    GradPlan grad;
    int32_t pitch;
    float *sums = nullptr, *part = nullptr;

    static int first_form(kfac_dtype_t dtype, kfac_dtype_t dpre_dtype) {
        return dtype == KFAC_F32 ? kProdParts : dpre_dtype == KFAC_F32 ? kProdMixed : kProdWide;
    }
    // dpre_dtype: KFAC_F32 or `dtype`
    GatedSpace(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype, kfac_dtype_t dpre_dtype, bool backward, void* base,
               bool input = false, bool weight = false)
        : ws(base), x(rows, d, dtype, ws), w(2 * width, d, dtype, ws), dpre(backward ? rows : 0, 2 * width, dpre_dtype, ws),
          size{!backward           ? ProdSize{rows, width, x.pitch, true}
               : input && rows > 0 ? ProdSize{rows, d, 2 * width}
                                   : ProdSize{},
               weight ? ProdSize{2 * width, d, rows} : ProdSize{}},
          plan(size, first_form(dtype, dpre_dtype), dtype == KFAC_BF16 && dpre_dtype == KFAC_BF16 ? kProdDeep : first_form(dtype, dpre_dtype)),
          grad(rows, width, dtype), pitch(norm_pitch(width)) {
        if (backward) sums = ws.take<float>((size_t)grad.parts * 2 * (size_t)pitch * sizeof(float));
        part = ws.take<float>(plan.part_bytes);
    }
};

// The kernel for few rows serves these calls where it is the faster by what it
// was measured to take, in us: for each round of a workgroup on every compute
// unit, `once` and `each` for a unit of 64 bytes of a wave's share of a row
// (bfloat16 of odd width, whose rows begin between words: three times that).
// Few rows / tiled, bfloat16, 1024 -> 4096: 1 row 5.4 / 12.6, 64 9.2 / 13.7, 128
// 15.9 / 14.2; 4608 -> 2304: 1 14.2 / 18.3, 64 34.5 / 20.2; 768 -> 768: 256
// 10.1 / 12.3, 512 18.3 / 12.6; 2305 -> 501: 1 20.1 / 16.2.  float32, which it
// reads without splitting it: 1024 -> 4096: 64 20.5 / 40.6, 256 69 / 50; 4608 ->
// 2304: 64 62 / 73, 128 112 / 77; 4096 -> 116: 1 18.6 / 21.1, 32 31 / 23.
constexpr int64_t kFewRows = 4096;   // at most
double few_rows_time(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype) {
    static constexpr double kOnce[2][3] = {{2.5, 3.0, 5.0}, {1.5, 2.2, 3.2}}, kEach[2][3] = {{0.8, 1.05, 2.0}, {0.65, 1.05, 1.55}};
    const bool bf16 = dtype == KFAC_BF16;
    const int blocks = gated_rows_blocks(rows), at = blocks == 1 ? 0 : blocks == 2 ? 1 : 2;
    const int64_t groups = ceil_div(width, 16) * ceil_div(rows, 16 * blocks), each = ceil_div(d, (bf16 ? 32 : 16) * kRowsWaves);
    const double unit = kEach[bf16][at] * (bf16 && d % 2 != 0 ? 3.0 : 1.0);
    return 2.0 + (double)ceil_div(groups, 256) * (kOnce[bf16][at] + unit * (double)each);
}

bool few_rows(const GatedSpace& s, int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype) {
    const bool bf16 = dtype == KFAC_BF16;
    // repacking: a launch, and its bytes (which stay in the caches)
    const double repack = s.x.repack ? 3.0 + (double)((rows + 2 * width) * d) * (bf16 ? 4.0 : 10.0) / 8e6 : 0.0;
    return rows <= kFewRows && few_rows_time(rows, d, width, dtype) <= s.plan.time + repack;
}

bool gated_act(int act) { return act >= kActSilu && act <= kActSigmoid; }

// A tensor of n elements of `dtype`, at least aligned to `least` bytes.
bool gated_tensor(const void* p, int64_t n, kfac_dtype_t dtype, size_t least) {
    return n == 0 || (p != nullptr && aligned(p, std::max(least, size_of(dtype))));
}

kfac_status_t gated_backward(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype, int act, const void* dh, const void* x,
                             const void* weight, const void* pre, void* dpre, kfac_dtype_t dpre_dtype, void* dx, void* dweight,
                             kfac_dtype_t dweight_dtype, float* dbias, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    if (!gated_shape(rows, d, width, dtype) || !gated_act(act) ||
        (dweight_dtype != KFAC_F32 && dweight_dtype != dtype) || !gated_tensor(dh, rows, dtype, 0) ||
        !gated_tensor(pre, rows, dtype, 0) || !gated_tensor(dpre, rows, dpre_dtype, 4) ||
        (dweight != nullptr && !gated_tensor(x, rows, dtype, 4)) ||
        (dx != nullptr && (!gated_tensor(dx, rows, dtype, 0) || !gated_tensor(weight, 1, dtype, 4))) ||
        !aligned(dweight, size_of(dweight_dtype)) || !aligned(dbias, 4))
        return KFAC_ERR_INVALID_VALUE;
    GatedSpace s(rows, d, width, dtype, dpre_dtype, true, workspace, dx != nullptr, dweight != nullptr);
    const kfac_status_t space = enough_space(workspace, workspace_bytes, s.ws.used);
    if (space != KFAC_OK) return space;
    const bool bf16 = dtype == KFAC_BF16, products = dx != nullptr || dweight != nullptr;
    const PairPlan& plan = s.plan;
    if (!plan.fits() || s.grad.parts > 65535) return KFAC_ERR_UNSUPPORTED;
    s.x.src = x;
    s.w.src = weight;
    s.dpre.src = dpre;
    RepackTable t{};
    int64_t blocks = 0;
    if (dx != nullptr && rows > 0) s.w.enter(t, blocks);
    if (dweight != nullptr) s.x.enter(t, blocks);
    if (blocks > kMaxThreads / 256) return KFAC_ERR_UNSUPPORTED;
    hipError_t e = blocks > 0 ? launch_repack(t, blocks, stream) : hipSuccess;
    if (e == hipSuccess && rows > 0) {
        GatedGradArgs g{};
        g.dh = dh;
        g.pre = pre;
        g.dpre = dpre;
        g.part = dbias != nullptr ? s.sums : nullptr;
        g.planes = products ? s.dpre.packed : nullptr;   // (none for bfloat16 dpre)
        g.plane = s.dpre.plane();
        g.plane_pitch = s.dpre.pitch;
        g.rows = rows;
        g.chunk = s.grad.chunk;
        g.width = (int32_t)width;
        g.pitch = s.pitch;
        g.act = act;
        e = launch_gated_grad(g, (int)s.grad.parts, bf16, dpre_dtype == KFAC_BF16, stream);
    }
    ProdPair pair{};
    const ProdForm& form = kProdForms[plan.form];
    for (int k = 0; k < 2; ++k) {
        ProdArgs& a = pair.p[k];
        const ProdSize& size = s.size[k];
        a.M = (int32_t)size.M;
        a.N = (int32_t)size.N;
        a.K = size.K;
        a.kchunk = plan.kchunk[k];
        a.tiles_m = (int32_t)size.tiles_m(form);
        a.tiles_n = (int32_t)size.tiles_n(form);
        a.tiles = (int32_t)plan.tiles[k];
        a.whole = (int32_t)plan.whole[k];
        a.splits = (int32_t)plan.splits[k];
        a.a = s.dpre.operand(k == 0 ? (int32_t)rows : (int32_t)(2 * width));
        a.b = (k == 0 ? s.w : s.x).operand((int32_t)d);
        a.out_bf16 = k == 0 ? bf16 : dweight_dtype == KFAC_BF16;
        a.out = k == 0 ? dx : dweight;
    }
    // dx's shares, then dW's
    pair.p[0].part = s.part;
    pair.p[1].part = s.part + (size_t)(plan.tiles[0] - plan.whole[0]) * (size_t)plan.splits[0] * (size_t)(form.m * form.n);
    if (e == hipSuccess && plan.items() > 0) e = launch_gated_backward(pair, plan.form, plan.items(), stream);
    PartSums sums{};
    if (dbias != nullptr) {
        sums.part = s.sums;
        sums.parts = (int32_t)s.grad.parts;
        sums.pitch = s.pitch;
        sums.d = (int32_t)width;
        sums.dweight = dbias;
        sums.dbias = dbias + width;
    }
    if (e == hipSuccess) e = launch_gated_finish(pair, plan.form, sums, stream);
    return hip_status(e);
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" {

// ------------------------------------------------------------- layer norm --

kfac_status_t kfac_layer_norm_forward(int64_t rows, int64_t d, kfac_dtype_t dtype, const void* x, int64_t x_stride, void* y,
                                      int64_t y_stride, float* mean, float* rstd, const void* weight, const void* bias,
                                      kfac_dtype_t weight_dtype, float eps, hipStream_t stream) {
    if (!norm_shape(rows, d) || !norm_types(dtype, weight_dtype) || !norm_rows(x, x_stride, rows, d, dtype) ||
        !norm_rows(y, y_stride, rows, d, dtype) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !norm_vector(weight, weight_dtype) || !norm_vector(bias, weight_dtype) || !(eps >= 0.0f) || !std::isfinite(eps))
        return KFAC_ERR_INVALID_VALUE;
    if (rows == 0) return KFAC_OK;
    NormArgs a{};
    a.x = x;
    a.y = y;
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    a.mean = mean;
    a.rstd = rstd;
    a.weight = weight;
    a.bias = bias;
    a.rows = rows;
    a.d = (int32_t)d;
    a.eps = eps;
    return hip_status(launch_norm_forward(a, dtype == KFAC_BF16, weight_dtype == KFAC_BF16, stream));
}

size_t kfac_layer_norm_workspace_size(int64_t rows, int64_t d) { return norm_shape(rows, d) ? norm_ws(rows, d) : SIZE_MAX; }

kfac_status_t kfac_layer_norm_backward(int64_t rows, int64_t d, kfac_dtype_t dtype, const void* dy, int64_t dy_stride,
                                       const void* x, int64_t x_stride, const float* mean, const float* rstd,
                                       const void* weight, void* dx, int64_t dx_stride, void* dweight, void* dbias,
                                       kfac_dtype_t weight_dtype, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
    if (!norm_shape(rows, d) || !norm_types(dtype, weight_dtype) || !norm_rows(dy, dy_stride, rows, d, dtype) ||
        !norm_rows(x, x_stride, rows, d, dtype) || (dx != nullptr && !norm_rows(dx, dx_stride, rows, d, dtype)) ||
        (rows > 0 && (mean == nullptr || rstd == nullptr)) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !norm_vector(weight, weight_dtype) || !norm_vector(dweight, weight_dtype) || !norm_vector(dbias, weight_dtype))
        return KFAC_ERR_INVALID_VALUE;
    const bool sums = dweight != nullptr || dbias != nullptr;
    const kfac_status_t space = enough_space(workspace, workspace_bytes, sums ? norm_ws(rows, d) : 0);
    if (space != KFAC_OK) return space;
    NormArgs a{};
    PartSums p{};
    a.x = x;
    a.dy = dy;
    a.y = dx;
    a.x_stride = x_stride;
    a.dy_stride = dy_stride;
    a.y_stride = dx_stride;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.weight = weight;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    a.rows = rows;
    a.d = (int32_t)d;
    a.pitch = norm_pitch(d);
    a.parts = (int32_t)norm_parts(rows, d, dtype == KFAC_BF16);
    hipError_t e = hipSuccess;
    if (rows > 0 && (sums || dx != nullptr)) e = launch_norm_backward(a, dtype == KFAC_BF16, weight_dtype == KFAC_BF16, stream);
    p.part = a.part;
    p.dweight = dweight;
    p.dbias = dbias;
    p.d = a.d;
    p.pitch = a.pitch;
    p.parts = a.parts;
    if (e == hipSuccess && sums) e = launch_norm_sums(p, weight_dtype == KFAC_BF16, stream);
    return hip_status(e);
}

// ------------------------------------------------------------------ gated --

size_t kfac_gated_workspace_size(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype, int backward) {
    if (!gated_shape(rows, d, width, dtype)) return SIZE_MAX;
    if (!backward) {
        const GatedSpace s(rows, d, width, dtype, dtype, false, nullptr);
        return few_rows(s, rows, d, width, dtype) ? 0 : s.ws.used;
    }
    // of both products together, or of one alone
    size_t most = 0;
    for (int k = 1; k < 4; ++k)
        most = std::max(most, GatedSpace(rows, d, width, dtype, backward == 2 ? KFAC_F32 : dtype, true, nullptr, (k & 1) != 0,
                                         (k & 2) != 0).ws.used);
    return most;
}

kfac_status_t kfac_gated_forward(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype, kfac_act_t act, const void* x,
                                 const void* weight, const float* bias, void* h, void* pre, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    if (!gated_shape(rows, d, width, dtype) || !gated_act(act) || !gated_tensor(x, rows * d, dtype, 4) ||
        !gated_tensor(weight, 1, dtype, 4) || !aligned(bias, 4) || !gated_tensor(h, rows, dtype, 0) ||
        (pre != nullptr && !gated_tensor(pre, rows, dtype, 0)))
        return KFAC_ERR_INVALID_VALUE;
    if (rows == 0) return KFAC_OK;
    GatedSpace s(rows, d, width, dtype, dtype, false, workspace);
    if (few_rows(s, rows, d, width, dtype)) {
        RowsArgs r{};
        r.x = x;
        r.weight = weight;
        r.bias = bias;
        r.h = h;
        r.pre = pre;
        r.rows = rows;
        r.d = (int32_t)d;
        r.width = (int32_t)width;
        r.act = act;
        return hip_status(launch_gated_rows(r, dtype == KFAC_BF16, stream));
    }
    const kfac_status_t space = enough_space(workspace, workspace_bytes, s.ws.used);
    if (space != KFAC_OK) return space;
    const PairPlan& plan = s.plan;
    const ProdForm& form = kProdForms[plan.form];
    ProdArgs a{};
    if (!plan.fits()) return KFAC_ERR_UNSUPPORTED;
    s.x.src = x;
    s.w.src = weight;
    RepackTable t{};
    int64_t blocks = 0;
    s.x.enter(t, blocks);
    s.w.enter(t, blocks);
    if (blocks > kMaxThreads / 256) return KFAC_ERR_UNSUPPORTED;
    if (blocks > 0 && launch_repack(t, blocks, stream) != hipSuccess) return KFAC_ERR_HIP;
    a.M = (int32_t)rows;
    a.N = (int32_t)width;
    a.K = s.size[0].K;
    a.kchunk = plan.kchunk[0];
    a.tiles_m = (int32_t)s.size[0].tiles_m(form);
    a.tiles_n = (int32_t)s.size[0].tiles_n(form);
    a.tiles = (int32_t)plan.tiles[0];
    a.whole = (int32_t)plan.whole[0];
    a.splits = (int32_t)plan.splits[0];
    a.part = s.part;
    a.a = s.x.operand((int32_t)rows);
    a.b = s.w.operand((int32_t)width, (int32_t)width);
    a.width = (int32_t)width;
    a.act = act;
    a.out_bf16 = dtype == KFAC_BF16;
    a.bias = bias;
    a.out = h;
    a.pre = pre;
    hipError_t e = launch_gated_forward(a, plan.form, plan.items(), stream);
    if (e == hipSuccess && a.whole < a.tiles) e = launch_gated_forward_finish(a, plan.form, stream);
    return hip_status(e);
}

kfac_status_t kfac_gated_backward(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype, kfac_act_t act, const void* dh,
                                  const void* x, const void* weight, const void* pre, void* dpre, void* dx, void* dweight,
                                  kfac_dtype_t dweight_dtype, float* dbias, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
    return gated_backward(rows, d, width, dtype, act, dh, x, weight, pre, dpre, dtype, dx, dweight, dweight_dtype, dbias,
                          workspace, workspace_bytes, stream);
}

kfac_status_t kfac_gated_backward_f32(int64_t rows, int64_t d, int64_t width, kfac_act_t act, const void* dh, const void* x,
                                      const void* weight, const void* pre, float* dpre, void* dx, void* dweight,
                                      kfac_dtype_t dweight_dtype, float* dbias, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
    return gated_backward(rows, d, width, KFAC_BF16, act, dh, x, weight, pre, dpre, KFAC_F32, dx, dweight, dweight_dtype, dbias,
                          workspace, workspace_bytes, stream);
}

// --------------------------------------------------------- gradient norm --

size_t kfac_grad_norm_workspace_size(int n) { return n >= 1 && n <= KFAC_MAX_COUNT ? clip_ws(n) : SIZE_MAX; }

kfac_status_t kfac_grad_norm(int n, const void* const* g, const int64_t* count, const kfac_dtype_t* dtype, float* norm,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int64_t chunks;
    if (!clip_tensors(n, g, count, dtype, chunks) || norm == nullptr || !aligned(norm, 4)) return KFAC_ERR_INVALID_VALUE;
    const kfac_status_t space = enough_space(workspace, workspace_bytes, clip_ws(n));
    if (space != KFAC_OK) return space;
    ClipTable t{};
    const kfac_status_t st = clip_squares(n, g, count, dtype, chunks, norm, workspace, t, stream);
    return st != KFAC_OK ? st : hip_status(launch_clip_norm(t, stream));
}

kfac_status_t kfac_grad_clip(int n, const void* const* g, void* const* out, const int64_t* count, const kfac_dtype_t* dtype,
                             float max_norm, float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int64_t chunks, same;
    if (!clip_tensors(n, g, count, dtype, chunks) || !clip_tensors(n, out, count, dtype, same) || norm == nullptr ||
        !aligned(norm, 4) || !(max_norm >= 0.0f) || !clip_apart(n, g, out, count, dtype, norm))
        return KFAC_ERR_INVALID_VALUE;
    const kfac_status_t space = enough_space(workspace, workspace_bytes, clip_ws(n));
    if (space != KFAC_OK) return space;
    ClipTable t{};
    const kfac_status_t st = clip_squares(n, g, count, dtype, chunks, norm, workspace, t, stream);
    if (st != KFAC_OK) return st;
    if (chunks == 0) return hip_status(launch_clip_norm(t, stream));
    int64_t bytes = 0;
    for (int i = 0; i < n; ++i) bytes += count[i] * (int64_t)size_of(dtype[i]);
    t.max_norm = max_norm;
    t.writes_norm = 1;
    t.once = bytes > kLastCache;   // what outgrows the last cache is scaled past it
    // the last tables first: the caches may still hold their tensors
    int16_t first[KFAC_MAX_COUNT / kClipGroup + 2];
    int groups = 0;
    for (int i = 0; i < n; ++groups) {
        first[groups] = (int16_t)i;
        for (int taken = 0; i < n && taken < kClipGroup; ++i) taken += count[i] > 0;
    }
    for (int k = groups - 1; k >= 0; --k) {
        clip_table(first[k], n, g, out, count, dtype, t);
        if (t.n == 0) continue;
        if (launch_clip_scale(t, clip_parts(t.chunks, chunks), stream) != hipSuccess) return KFAC_ERR_HIP;
        t.writes_norm = 0;
    }
    return KFAC_OK;
}

}  // extern "C"
