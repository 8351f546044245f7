// Layer norm over the rows of a matrix, forward and backward.
//
//   mean = sum x / d, rstd = (sum (x - mean)^2 / d + eps)^-1/2
//   xh = (x - mean) rstd,  y = weight xh + bias
//   a = weight dy,  dx = rstd (a - mean(a) - xh mean(a xh))
//   dweight = sum over rows of dy xh,  dbias = sum over rows of dy
//
// Memory bounds both: a row is read once and stays in registers, so that the
// variance is summed around the mean (no cancellation) at no further traffic.
// A wave takes a row of 257 to 1024 elements, or two to eight shorter ones;
// three to sixteen waves take a longer one.  A workgroup keeps its part of the
// weights and goes from row to row, the next one on its way.  Backward, it adds up dy xh and dy of its rows in
// registers and leaves the sums in the workspace; a second launch adds the
// workgroups' sums in a fixed order.  Statistics and sums are float32.
//
// Measured (medians of a kernel trace, rows from memory; backward: both
// launches): 25088 x 2305 float32 backward 130 us (5.3 TB/s), 25088 x 1024 bfloat16
// forward 20 (5.1 TB/s) and backward 33; 4096 x 1024 7.8 and 12.9, where a wave
// has one or two rows and their latency bounds it; 8192 x 16384 float32 backward
// 347 (4.6 TB/s: of the 128 registers that 16 waves leave a lane 13 spill; 8192 x
// 8192 169).
#include <algorithm>

#include "encoder.h"
#include "encoder_common.h"

namespace kfac {
namespace {

// Waves at work on a compute unit.  25088 rows of 2304, forward in bfloat16 and
// float32: 16 waves 66 and 89 us, 24 58 and 89, 32 69 and 97; backward,
// where each workgroup leaves sums to add: 8 waves 120 and 138 us, 12 89 and
// 127, 16 75 and 149, 24 75 and 154.
constexpr int kForwardWaves = 24, kBackwardWaves = 16, kBackwardWavesF32 = 12;

constexpr int threads_of(int W) { return W == 1 ? 256 : 64 * W; }

// L lanes of a wave, or the lanes of up to W waves, hold a row: of `lanes`
// lanes, vector n of lane t is the row's n lanes + t th.
template <typename T, int W, int L, int E, bool SHORT>
struct RowOf {
    static constexpr int N = Vec<T>::N, NV = E / N;
    static constexpr int ROWS = W == 1 ? 256 / L : 1;   // per workgroup
    static __device__ __forceinline__ int lanes() { return W == 1 ? L : (int)blockDim.x; }
    // this wave's first row of the workgroup's, this thread's of its wave's, and its lane of the row
    static __device__ __forceinline__ int wave_row() {
        return W == 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) * (64 / L) : 0;
    }
    static __device__ __forceinline__ int row() { return L < 64 ? (int)(threadIdx.x & 63) / L : 0; }
    static __device__ __forceinline__ int lane() { return W == 1 ? (int)threadIdx.x % L : (int)threadIdx.x; }
    static __device__ __forceinline__ int at(int n, int t) { return (n * lanes() + t) * N; }

    // A row on its way: of S, which may be the wider type.
    template <typename S>
    struct Row {
        static constexpr int M = Vec<S>::N, K = E / M;
        RowVec<S, SHORT> v[K];
        __device__ __forceinline__ void get(const S* p, int d, int t) {
#pragma unroll
            for (int k = 0; k < K; ++k) v[k].get(p, at(k * M / N, t) + k * M % N, d);
        }
        __device__ __forceinline__ void open(float (&x)[E]) const {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float q[M];
                v[k].open(q);
#pragma unroll
                for (int e = 0; e < M; ++e) x[k * M + e] = q[e];
            }
        }
    };
    static __device__ __forceinline__ void store(T* p, const float (&v)[E], int d, int t) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float q[N];
#pragma unroll
            for (int e = 0; e < N; ++e) q[e] = v[n * N + e];
            store_some<T>(p + at(n, t), q, d - at(n, t));
        }
    }
    // which elements exist
    static __device__ __forceinline__ bool in(int i, int d, int t) { return at(i / N, t) + i % N < d; }
};

// Sums over the lanes of a row, in every one of them.  A place is written again
// two calls later: every wave has passed the call between, and so has read it.
template <int W, int L, int K>
__device__ __forceinline__ void row_sums(float (&s)[K], float (*place)[W], int wave) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = lane_sum<L>(s[k]);
    if constexpr (W > 1) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((threadIdx.x & 63) == 0) place[k][wave] = s[k];
        lds_barrier();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            s[k] = place[k][0];
            for (int w = 1; w < (int)blockDim.x / 64; ++w) s[k] += place[k][w];
        }
    }
}

template <typename T, typename S, int W, int L, int E, bool SHORT>
__global__ __launch_bounds__(threads_of(W)) void norm_forward_kernel(NormArgs A) {
    using R = RowOf<T, W, L, E, SHORT>;
    __shared__ float places[2][1][W];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int t = R::lane(), d = A.d;
    const float inv = 1.0f / (float)d;
    float w[E], b[E];
    {
        typename R::template Row<S> rw, rb;
        if (A.weight) rw.get(static_cast<const S*>(A.weight), d, t);
        if (A.bias) rb.get(static_cast<const S*>(A.bias), d, t);
        if (A.weight) rw.open(w);
        if (A.bias) rb.open(b);
    }
    const int64_t step = (int64_t)gridDim.x * R::ROWS;
    // the next row is on its way while this one is summed (past the last: that one again)
    typename R::template Row<T> rx;
    auto fetch = [&](int64_t row) { rx.get(static_cast<const T*>(A.x) + min(row, A.rows - 1) * A.x_stride, d, t); };
    const int64_t first = (int64_t)blockIdx.x * R::ROWS + R::wave_row();
    fetch(first + R::row());
    for (int64_t turn = first; turn < A.rows; turn += step) {
        const int64_t row = turn + R::row();
        float x[E];
        rx.open(x);
        fetch(row + step);
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] += x[i];
        row_sums<W, L>(s, places[0], wave);
        const float mean = s[0] / (float)d;   // a row of one number has it as its mean
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            x[i] = R::in(i, d, t) ? x[i] - mean : 0.0f;
            s[0] += x[i] * x[i];
        }
        row_sums<W, L>(s, places[1], wave);
        const float rstd = 1.0f / sqrtf(s[0] * inv + A.eps);
        if (L < 64 && row >= A.rows) continue;
        if (t == 0) {
            if (A.mean) *as_global(A.mean + row) = mean;
            if (A.rstd) *as_global(A.rstd + row) = rstd;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            x[i] *= rstd;
            if (A.weight) x[i] *= w[i];
            if (A.bias) x[i] += b[i];
        }
        R::store(static_cast<T*>(A.y) + row * A.y_stride, x, d, t);
    }
}

template <typename T, typename S, int W, int L, int E, bool SHORT>
__global__ __launch_bounds__(threads_of(W)) void norm_backward_kernel(NormArgs A) {
    using R = RowOf<T, W, L, E, SHORT>;
    __shared__ float places[2][2][W];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int t = R::lane(), d = A.d;
    const float inv = 1.0f / (float)d;
    float w[E], dw[E], db[E];
    if (A.weight) {
        typename R::template Row<S> rw;
        rw.get(static_cast<const S*>(A.weight), d, t);
        rw.open(w);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = 1.0f;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.0f;
    const int64_t step = (int64_t)gridDim.x * R::ROWS;
    int turn = 0;
    // the next row is on its way while this one is summed, where the registers hold both
    constexpr bool AHEAD = W < 16 || E < 16;
    typename R::template Row<T> rx, rdy;
    float next_mean = 0.0f, next_rstd = 0.0f;
    auto fetch = [&](int64_t row) {
        row = min(row, A.rows - 1);
        rx.get(static_cast<const T*>(A.x) + row * A.x_stride, d, t);
        rdy.get(static_cast<const T*>(A.dy) + row * A.dy_stride, d, t);
        next_mean = *as_global(A.mean + row);
        next_rstd = *as_global(A.rstd + row);
    };
    const int64_t first = (int64_t)blockIdx.x * R::ROWS + R::wave_row();
    if (AHEAD) fetch(first + R::row());
    for (int64_t base = first; base < A.rows; base += step, turn ^= 1) {
        const int64_t row = base + R::row();
        const bool there = L == 64 || row < A.rows;
        float x[E], dy[E];
        if (!AHEAD) fetch(row);
        rx.open(x);
        rdy.open(dy);
        const float mean = next_mean, rstd = next_rstd;
        if (AHEAD) fetch(row + step);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            x[i] = there && R::in(i, d, t) ? (x[i] - mean) * rstd : 0.0f;   // dy is 0 past the row
            if (L < 64) dy[i] = there ? dy[i] : 0.0f;
            dw[i] += dy[i] * x[i];
            db[i] += dy[i];
            dy[i] *= w[i];
            s[0] += dy[i];
            s[1] += dy[i] * x[i];
        }
        if (A.y == nullptr) continue;
        row_sums<W, L>(s, places[turn], wave);
        const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < E; ++i) dy[i] = rstd * (dy[i] - m0 - x[i] * m1);
        if (there) R::store(static_cast<T*>(A.y) + row * A.y_stride, dy, d, t);
    }
    if (A.part == nullptr) return;
    float* part = A.part + (int64_t)blockIdx.x * 2 * A.pitch;
    if constexpr (R::ROWS > 1) {
        // the rows of a wave, then the waves in order
        constexpr int COLUMNS = L * E;
        __shared__ __attribute__((aligned(16))) float sums[4][2][COLUMNS];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            dw[i] = column_sum<L>(dw[i]);
            db[i] = column_sum<L>(db[i]);
        }
        if ((int)(threadIdx.x & 63) < L) {
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                const int at = R::at(i / R::N, t) + i % R::N;
                *reinterpret_cast<uint4v*>(&sums[wave][0][at]) = Vec<float>::close({dw[i], dw[i + 1], dw[i + 2], dw[i + 3]});
                *reinterpret_cast<uint4v*>(&sums[wave][1][at]) = Vec<float>::close({db[i], db[i + 1], db[i + 2], db[i + 3]});
            }
        }
        lds_barrier();
#pragma unroll
        for (int k = 0; k < 2; ++k)
            for (int c = threadIdx.x; c < d; c += 256)
                *as_global(part + k * A.pitch + c) = ((sums[0][k][c] + sums[1][k][c]) + sums[2][k][c]) + sums[3][k][c];
    } else {
#pragma unroll
        for (int n = 0; n < R::NV; ++n)
#pragma unroll
            for (int k = 0; k < R::N; k += 4) {
                float p[4], q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = dw[n * R::N + k + e];
                    q[e] = db[n * R::N + k + e];
                }
                const int at = R::at(n, t) + k;
                store_some<float>(part + at, p, d - at);
                store_some<float>(part + A.pitch + at, q, d - at);
            }
    }
}

template <typename S>
__global__ __launch_bounds__(256) void norm_sums_kernel(PartSums A) {
    __shared__ float join[4][kSumColumns];
    add_parts<S>(A, blockIdx.x, join);
}

// Waves of a row of d elements, and of a workgroup: 8 elements a lane (one
// wave holds up to 1024), past kForwardWide or kBackwardWide elements 16.
// Rows of 2304 bfloat16 elements, 25088 of them, backward: 97 us by four waves
// of 16 elements a lane, most of whose second vectors lie past the row, 79 by
// five waves of 8.  25088 of 8000, forward: 258 by sixteen waves of 8, 182 by
// eight of 16; 8192 of 5000: 45 either way; backward 6500 wide 86 and 96.
constexpr int64_t kForwardWide = 6144, kBackwardWide = 8192;
int norm_waves(int64_t d, bool backward) {
    return d <= 1024 ? 1 : (int)(d <= (backward ? kBackwardWide : kForwardWide) ? (d + 511) / 512 : (d + 1023) / 1024);
}

// Lanes of a row of one wave, of 8 elements each (16 past 512).  Rows of 64
// bfloat16 elements, 200000 of them, by 8 lanes each: 13.7 us forward, 22.8
// backward (61 and 86 with a wave for each row); 100000 of 256 by 32: 23.6 and
// 35.6 (36.3 and 51.4).
int norm_lanes(int64_t d) { return d <= 64 ? 8 : d <= 128 ? 16 : d <= 256 ? 32 : 64; }

template <typename T, typename S, int W, int L, int E, bool SHORT>
hipError_t launch_form(const NormArgs& a, bool backward, hipStream_t stream) {
    using R = RowOf<T, W, L, E, SHORT>;
    const dim3 block((unsigned)(W == 1 ? 256 : 64 * norm_waves(a.d, backward)));
    if (backward) {
        hipLaunchKernelGGL((norm_backward_kernel<T, S, W, L, E, SHORT>), dim3((unsigned)a.parts), block, 0, stream, a);
    } else {
        const int64_t blocks = (a.rows + R::ROWS - 1) / R::ROWS, most = 256 * std::max(1, kForwardWaves / std::max(4, norm_waves(a.d, false)));
        hipLaunchKernelGGL((norm_forward_kernel<T, S, W, L, E, SHORT>), dim3((unsigned)std::min(blocks, most)), block, 0, stream, a);
    }
    return hipGetLastError();
}

template <typename T, typename S>
hipError_t launch_typed(const NormArgs& a, bool backward, hipStream_t stream) {
    if (a.d < 8) return launch_form<T, S, 1, 8, 8, true>(a, backward, stream);
    if (a.d <= 64) return launch_form<T, S, 1, 8, 8, false>(a, backward, stream);
    if (a.d <= 128) return launch_form<T, S, 1, 16, 8, false>(a, backward, stream);
    if (a.d <= 256) return launch_form<T, S, 1, 32, 8, false>(a, backward, stream);
    if (a.d <= 512) return launch_form<T, S, 1, 64, 8, false>(a, backward, stream);
    if (a.d <= 1024) return launch_form<T, S, 1, 64, 16, false>(a, backward, stream);
    if (a.d <= 2048) return launch_form<T, S, 4, 64, 8, false>(a, backward, stream);
    if (a.d <= 4096) return launch_form<T, S, 8, 64, 8, false>(a, backward, stream);
    if (a.d <= (backward ? kBackwardWide : kForwardWide)) return launch_form<T, S, 16, 64, 8, false>(a, backward, stream);
    return launch_form<T, S, 16, 64, 16, false>(a, backward, stream);
}

hipError_t launch_any(const NormArgs& a, bool bf16, bool weight_bf16, bool backward, hipStream_t stream) {
    if (!bf16) return launch_typed<float, float>(a, backward, stream);
    if (!weight_bf16) return launch_typed<__bf16, float>(a, backward, stream);
    return launch_typed<__bf16, __bf16>(a, backward, stream);
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t d, bool bf16) {
    const int waves = norm_waves(d, true), all = bf16 ? kBackwardWaves : kBackwardWavesF32;
    // rows of a wave or less: 4 to 32 to a workgroup of four waves, two workgroups on a compute unit (three: 4096 x
    // 1024 bfloat16 12.6 to 14.3 us)
    const int per = 256 / norm_lanes(d);
    const int64_t blocks = waves == 1 ? (rows + per - 1) / per : rows, most = waves == 1 ? 512 : 256 * std::max(1, all / waves);
    return std::min(blocks, most);
}

hipError_t launch_norm_forward(const NormArgs& a, bool bf16, bool weight_bf16, hipStream_t stream) {
    return launch_any(a, bf16, weight_bf16, false, stream);
}

hipError_t launch_norm_backward(const NormArgs& a, bool bf16, bool weight_bf16, hipStream_t stream) {
    return launch_any(a, bf16, weight_bf16, true, stream);
}

hipError_t launch_norm_sums(const PartSums& a, bool weight_bf16, hipStream_t stream) {
    const dim3 grid((unsigned)sums_blocks(a.pitch));
    if (weight_bf16) hipLaunchKernelGGL(norm_sums_kernel<__bf16>, grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(norm_sums_kernel<float>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace kfac
