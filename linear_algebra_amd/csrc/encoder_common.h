// Device helpers of the encoder layer's elementwise and row kernels.
#pragma once

#include "device_common.h"
#include "encoder.h"

namespace kfac {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
// 16 bytes at an address that need only hold one element
typedef uint32_t loose16 __attribute__((ext_vector_type(4), aligned(2)));

// 16 bytes of T as floats and back (bfloat16 rounded to nearest even).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void open(float (&v)[4], uint4v q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(q[e]);
    }
    static __device__ __forceinline__ uint4v close(const float (&v)[4]) {
        return uint4v{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    }
};
template <>
struct Vec<__bf16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void open(float (&v)[8], uint4v q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(q[e] << 16);
            v[2 * e + 1] = __uint_as_float(q[e] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4v close(const float (&v)[8]) {
        uint4v q;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            q[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(floatx2{v[2 * e], v[2 * e + 1]}, bf16x2));
        return q;
    }
};

// The elements [at, at + N) of a row of d elements, zeros past its end, without
// a branch (a load behind one is waited for where the branch ends, and no
// other load is then in flight): what reaches past the end is read so that it
// ends with the row, and shifted.  Rows of fewer than N elements (SHORT) are
// read one by one.  get() issues the load, open() waits for it.
template <typename T, bool SHORT>
struct RowVec {
    static constexpr int N = Vec<T>::N, ES = 16 / N;
    uint4v q;
    int shift;
    __device__ __forceinline__ void get(const T* row, int at, int d) {
        if constexpr (SHORT) {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (at + e >= d) continue;
                if constexpr (ES == 4) w[e] = __builtin_bit_cast(uint32_t, *as_global(row + at + e));
                else w[e / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, *as_global(row + at + e)) << (16 * (e & 1));
            }
            q = uint4v{w[0], w[1], w[2], w[3]};
            shift = 0;
        } else {
            const int pos = min(at, d - N);
            q = *(const __attribute__((address_space(1))) loose16*)(row + pos);
            shift = at - pos;
        }
    }
    // ends: whether any lane's vector may reach past the end (the same in all)
    __device__ __forceinline__ void open(float (&v)[N], bool ends = true) const { Vec<T>::open(v, raw(ends)); }
    __device__ __forceinline__ uint4v raw(bool ends) const {
        uint4v w = q;
        if (!SHORT && ends) {
            const int words = shift / (4 / ES);
            if (ES == 2) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = __builtin_amdgcn_alignbit(e < 3 ? w[e + 1] : 0u, w[e], (uint32_t)(shift & 1) * 16);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = words & 1 ? (e < 3 ? w[e + 1] : 0u) : w[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = words & 2 ? (e < 2 ? w[e + 2] : 0u) : w[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = shift >= N ? 0u : w[e];
        }
        return w;
    }
};

template <typename T>
__device__ __forceinline__ void store_all(T* p, const float (&v)[Vec<T>::N]) {
    *(__attribute__((address_space(1))) loose16*)p = Vec<T>::close(v);
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, const float (&v)[Vec<T>::N], int count) {
    constexpr int N = Vec<T>::N;
    if (count >= N) {
        store_all<T>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < count) *as_global(p + e) = (T)v[e];
    }
}

// A barrier that waits for the workgroup's LDS accesses only: loads and
// stores in flight stay so (__syncthreads() would wait for them too).
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
// The sum over a wave, in every lane: within rows of 16 lanes by moves beside
// the additions, then the four rows in order.
__device__ __forceinline__ float wave_sum(float x) {
    x += dpp<0xb1>(x);    // lanes 1 0 3 2 of each four
    x += dpp<0x4e>(x);    // lanes 2 3 0 1
    x += dpp<0x141>(x);   // mirrored halves of a row
    x += dpp<0x140>(x);   // mirrored rows
    auto row = [&](int lane) { return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(x), lane)); };
    return ((row(0) + row(16)) + row(32)) + row(48);
}

// x + the x of lane ^ 16 (its row of 16 lanes changed for the neighbouring one), or ^ 32.
__device__ __forceinline__ float add_row(float x) {
    const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(v[0]) + __uint_as_float(v[1]);
}
__device__ __forceinline__ float add_half(float x) {
    const auto v = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(v[0]) + __uint_as_float(v[1]);
}

// The sum over each L neighbouring lanes, in every one of them.
template <int L>
__device__ __forceinline__ float lane_sum(float x) {
    static_assert(L == 8 || L == 16 || L == 32 || L == 64, "lanes of a row");
    if constexpr (L == 64) return wave_sum(x);
    x += dpp<0xb1>(x);
    x += dpp<0x4e>(x);
    x += dpp<0x141>(x);
    if constexpr (L >= 16) x += dpp<0x140>(x);
    if constexpr (L >= 32) x = add_row(x);
    return x;
}

// The sum over the lanes that are multiples of L apart, in every one of them.
template <int L>
__device__ __forceinline__ float column_sum(float x) {
    if constexpr (L <= 8) x += dpp<0x128>(x);   // rows of 16 turned by 8
    if constexpr (L <= 16) x = add_row(x);
    if constexpr (L <= 32) x = add_half(x);
    return x;
}

// Adds the sums of many workgroups, [parts][2][pitch]: kSumColumns columns of
// one of the two by a workgroup of 256 threads, 32 groups of parts of four
// columns a thread, the groups joined in a fixed order.
template <typename S>
__device__ __forceinline__ void add_parts(const PartSums& A, int block, float (*join)[kSumColumns]) {
    constexpr int LANES = kSumColumns / 4, GROUPS = 256 / LANES;
    const int c = 4 * (threadIdx.x % LANES), g = threadIdx.x / LANES;
    const int per = (A.pitch + kSumColumns - 1) / kSumColumns;
    const int which = block / per, first = block % per * kSumColumns, at = first + c;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (at < A.pitch) {
        const float* p = A.part + which * A.pitch + at;
        const int64_t step = 2 * (int64_t)A.pitch;
#pragma unroll 8
        for (int k = g; k < A.parts; k += GROUPS) {
            float q[4];
            Vec<float>::open(q, *as_global(reinterpret_cast<const uint4v*>(p + k * step)));
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += q[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = column_sum<LANES>(s[e]);
    if ((threadIdx.x & 63) < LANES)
#pragma unroll
        for (int e = 0; e < 4; ++e) join[threadIdx.x >> 6][c + e] = s[e];
    __syncthreads();
    if (threadIdx.x >= kSumColumns) return;
    const int col = first + threadIdx.x;
    const float v = ((join[0][threadIdx.x] + join[1][threadIdx.x]) + join[2][threadIdx.x]) + join[3][threadIdx.x];
    S* out = static_cast<S*>(which ? A.dbias : A.dweight);
    if (out != nullptr && col < A.d) *as_global(out + col) = (S)v;
}

}  // namespace kfac
