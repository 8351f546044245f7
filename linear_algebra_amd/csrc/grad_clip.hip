// The norm of many gradients taken together, and their scaling.
//
//   norm = sqrt(sum over all tensors of g^2)
//   out = c g,  c = min(1, max_norm / (norm + 1e-6))
//
// Memory bounds both passes.  Workgroups go through chunks of 8192 elements of
// whatever tensor they lie in, each with a sum of its own in float64 (a
// square of a float32 number neither overflows nor vanishes there, and the
// float64 units have the time), which the next launch adds up in a fixed
// order: every scaling workgroup by itself, at most some thousand numbers from
// the L2, instead of in a launch between.  The scaling runs backwards through
// the chunks, so that it begins with those that the caches still hold, and
// where the gradients outgrow the caches it reads and writes past them (its
// own would push out what it has yet to read).  151 million float32 gradients
// in 144 tensors: 300 us for 1.8 GB, 6.0 TB/s (through the caches 354).
#include <type_traits>

#include "encoder.h"
#include "encoder_common.h"

namespace kfac {
namespace {

constexpr int NT = kClipThreads;

// The tensor that holds a chunk: the last one that begins at or before it
// (tensors without elements have no chunk and begin where the next does).
__device__ __forceinline__ int find_tensor(const ClipTable& T, uint32_t chunk) {
    int lo = 0, hi = T.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (T.t[mid].begin <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// A chunk's place: elements [at, at + count) of a tensor.
struct ClipChunk {
    const ClipTensor& t;
    int64_t at;
    int count;
    bool bf16;
    __device__ __forceinline__ ClipChunk(const ClipTable& T, uint32_t chunk) : t(T.t[find_tensor(T, chunk)]) {
        const uint32_t end = &t - T.t + 1 < T.n ? (&t)[1].begin : T.chunks;
        at = (int64_t)(chunk - t.begin) * kClipChunk;
        count = chunk + 1 == end ? (int)(t.last & ~kClipBf16) : kClipChunk;
        bf16 = (t.last & kClipBf16) != 0;
    }
};

// The chunk's vectors in turn: a thread's loads of eight vectors, then
// f(values, element, how many) of each.  A tensor's last chunk is read the
// same way, apart from one that is shorter than a vector.
template <bool ONCE, typename E, typename F>
__device__ __forceinline__ void each_vector(const E* p, int count, F f) {
    constexpr int N = Vec<E>::N, VECS = kClipChunk / (NT * N);
    auto turn = [&](auto kind, int vecs) {
        RowVec<E, decltype(kind)::value> q[VECS];
#pragma unroll
        for (int k = 0; k < VECS; ++k)
            if (k < vecs) q[k].get(p, ((int)threadIdx.x + k * NT) * N, count);
#pragma unroll
        for (int k = 0; k < VECS; ++k) {
            if (k >= vecs) break;
            float v[N];
            const int at = ((int)threadIdx.x + k * NT) * N;
            q[k].open(v);
            f(v, at, count - at);
        }
    };
    if (count == kClipChunk) {
        uint4v q[VECS];
#pragma unroll
        for (int k = 0; k < VECS; ++k) {
            const auto* at = (const __attribute__((address_space(1))) loose16*)(p + ((int)threadIdx.x + k * NT) * N);
            if constexpr (ONCE) q[k] = __builtin_nontemporal_load(at);
            else q[k] = *at;
        }
#pragma unroll
        for (int k = 0; k < VECS; ++k) {
            float v[N];
            Vec<E>::open(v, q[k]);
            f(v, ((int)threadIdx.x + k * NT) * N, N);
        }
    } else if (count >= N) {
        turn(std::false_type(), (count + NT * N - 1) / (NT * N));
    } else {
        turn(std::true_type(), 1);
    }
}

template <bool ONCE, typename E>
__device__ __forceinline__ void put(E* p, const float (&v)[Vec<E>::N], int left) {
    if (ONCE && left >= Vec<E>::N) {
        const loose16 q = Vec<E>::close(v);
        __builtin_nontemporal_store(q, (__attribute__((address_space(1))) loose16*)p);
    } else {
        store_some<E>(p, v, left);
    }
}

// The workgroup's sum, in every thread.
__device__ __forceinline__ double block_sum(double x, double* place) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) place[threadIdx.x >> 6] = x;
    __syncthreads();
    x = place[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) x += place[w];
    return x;
}

__global__ __launch_bounds__(NT) void clip_squares_kernel(ClipTable T) {
    __shared__ double place[NT / 64];
    double sum = 0.0;
    for (uint32_t chunk = blockIdx.x; chunk < T.chunks; chunk += gridDim.x) {
        const ClipChunk C(T, chunk);
        auto add = [&](const auto& v, int, int) {   // what lies past the end reads as 0
            for (float x : v) sum = fma((double)x, (double)x, sum);
        };
        if (C.bf16) each_vector<false>(static_cast<const __bf16*>(C.t.g) + C.at, C.count, add);
        else each_vector<false>(static_cast<const float*>(C.t.g) + C.at, C.count, add);
    }
    sum = block_sum(sum, place);
    if (threadIdx.x == 0) *as_global(T.part + T.first_part + blockIdx.x) = sum;
}

// The norm from the workgroups' sums.
__device__ __forceinline__ double norm_of(const ClipTable& T, double* place) {
    double sum = 0.0;
    for (int k = threadIdx.x; k < T.parts; k += NT) sum += *as_global(T.part + k);
    return sqrt(block_sum(sum, place));
}

__global__ __launch_bounds__(NT) void clip_norm_kernel(ClipTable T) {
    __shared__ double place[NT / 64];
    const double norm = norm_of(T, place);
    if (threadIdx.x == 0) *as_global(T.norm) = (float)norm;
}

// ONCE: past the caches.
template <bool ONCE>
__global__ __launch_bounds__(NT) void clip_scale_kernel(ClipTable T) {
    __shared__ double place[NT / 64];
    const double norm = norm_of(T, place);
    if (T.writes_norm && blockIdx.x == 0 && threadIdx.x == 0) *as_global(T.norm) = (float)norm;
    const double ratio = (double)T.max_norm / (norm + 1e-6);
    const float c = ratio > 1.0 ? 1.0f : (float)ratio;   // (a norm that is no number stays one)
    for (uint32_t chunk = blockIdx.x; chunk < T.chunks; chunk += gridDim.x) {
        const ClipChunk C(T, T.chunks - 1 - chunk);
        if (c == 1.0f && C.t.out == C.t.g) continue;   // times 1, in place
        if (C.bf16) {
            __bf16* out = static_cast<__bf16*>(C.t.out) + C.at;
            each_vector<ONCE>(static_cast<const __bf16*>(C.t.g) + C.at, C.count, [&](float (&v)[8], int e, int left) {
                for (float& x : v) x *= c;
                put<ONCE>(out + e, v, left);
            });
        } else {
            float* out = static_cast<float*>(C.t.out) + C.at;
            each_vector<ONCE>(static_cast<const float*>(C.t.g) + C.at, C.count, [&](float (&v)[4], int e, int left) {
                for (float& x : v) x *= c;
                put<ONCE>(out + e, v, left);
            });
        }
    }
}

}  // namespace

hipError_t launch_clip_squares(const ClipTable& t, int blocks, hipStream_t stream) {
    hipLaunchKernelGGL(clip_squares_kernel, dim3((unsigned)blocks), dim3(NT), 0, stream, t);
    return hipGetLastError();
}

hipError_t launch_clip_norm(const ClipTable& t, hipStream_t stream) {
    hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(NT), 0, stream, t);
    return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipTable& t, int blocks, hipStream_t stream) {
    if (t.once) hipLaunchKernelGGL(clip_scale_kernel<true>, dim3((unsigned)blocks), dim3(NT), 0, stream, t);
    else hipLaunchKernelGGL(clip_scale_kernel<false>, dim3((unsigned)blocks), dim3(NT), 0, stream, t);
    return hipGetLastError();
}

}  // namespace kfac
