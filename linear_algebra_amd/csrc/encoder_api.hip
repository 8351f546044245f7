// Host side of the operators around an encoder layer's products (layer norm,
// gradient norm and clipping): argument validation, work planning and launch
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

size_t norm_ws(int64_t rows, int64_t d) { return (size_t)norm_parts(rows, d) * 2 * (size_t)norm_pitch(d) * sizeof(float); }

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
// is written lies apart from everything but the gradient it stands for.
bool clip_apart(int n, const void* const* g, void* const* out, const int64_t* count, const kfac_dtype_t* dtype) {
    Range r[2 * KFAC_MAX_COUNT];
    int m = 0;
    bool sorted = true;
    auto take = [&](const void* p, size_t bytes) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
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
    return true;
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
    a.x = x;
    a.dy = dy;
    a.y = dx;
    a.x_stride = x_stride;
    a.dy_stride = dy_stride;
    a.y_stride = dx_stride;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.weight = weight;
    a.dweight = dweight;
    a.dbias = dbias;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    a.rows = rows;
    a.d = (int32_t)d;
    a.pitch = norm_pitch(d);
    a.parts = (int32_t)norm_parts(rows, d);
    hipError_t e = hipSuccess;
    if (rows > 0 && (sums || dx != nullptr)) e = launch_norm_backward(a, dtype == KFAC_BF16, weight_dtype == KFAC_BF16, stream);
    if (e == hipSuccess && sums) e = launch_norm_sums(a, weight_dtype == KFAC_BF16, stream);
    return hip_status(e);
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
        !aligned(norm, 4) || !(max_norm >= 0.0f) || !clip_apart(n, g, out, count, dtype))
        return KFAC_ERR_INVALID_VALUE;
    const kfac_status_t space = enough_space(workspace, workspace_bytes, clip_ws(n));
    if (space != KFAC_OK) return space;
    ClipTable t{};
    const kfac_status_t st = clip_squares(n, g, count, dtype, chunks, norm, workspace, t, stream);
    if (st != KFAC_OK) return st;
    if (chunks == 0) return hip_status(launch_clip_norm(t, stream));
    t.max_norm = max_norm;
    t.writes_norm = 1;
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
