// Layer inputs kept in 8 bits between the forward and the backward pass, and
// the two products that use them: the factor A = x^T x / rows and the
// gradient [dW | db] = g^T [x | 1].
//
// Both products sum over rows, so a block shares its scale along the rows of
// one column: 32 consecutive rows, e4m3 codes and one power of two, next to
// one another in memory as the matrix cores take them.  A code times its
// power of two is exactly a bfloat16 number (4 significant bits), so the
// codes are converted on the way to the bf16 matrix cores without a rounding;
// float32 gradients enter as three exact bf16 parts.
#include <type_traits>

#include "device_common.h"
#include "training.h"

namespace kfac {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef short short2v __attribute__((ext_vector_type(2)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));

constexpr int NT = kKeepThreads;
constexpr uint32_t kOOB = 0x80000000u;

__device__ __forceinline__ int find_layer(const KeepLaunch& L, int64_t block) {
    int k = 0;
    while (k + 1 < L.n && L.layer[k + 1].block_begin <= block) ++k;
    return k;
}

// Exponent of a block: the least e >= kKeepMinExp with top <= 448 2^e, from
// the bits of the largest finite magnitude (448 = 1.75 2^8).
__device__ __forceinline__ int block_exp(uint32_t top) {
    const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, kKeepMinExp);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Codes of one column's 32 rows and its scale byte.  Infinities and NaN do
// not count for the scale and become NaN codes (an infinity's quotient is
// out of range, which the conversion turns into NaN).
__device__ __forceinline__ void encode(const float (&v)[32], uint4v (&code)[2], uint8_t& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        const uint32_t u = __float_as_uint(v[r]) & 0x7fffffffu;
        top = max(top, u < 0x7f800000u ? u : 0u);
    }
    const int e = block_exp(top);
    const float s = pow2(e);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        short2v c = {0, 0};
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[4 * w], v[4 * w + 1], s, false);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[4 * w + 2], v[4 * w + 3], s, true);
        code[w >> 2][w & 3] = __builtin_bit_cast(uint32_t, c);
    }
    scale = (uint8_t)(e + 127);
}

// Workgroups take runs of columns of one block of rows, one column per
// thread (two of bf16 inputs whose rows allow 4-byte accesses): a wave reads
// 256 bytes of each of the 32 rows and writes the columns' codes, 32 bytes
// each, next to one another.  The values stay in registers between the
// maximum and the conversion, so each is read once.
template <bool BF16, int COLS>
__device__ __forceinline__ void store_block(const KeepLayer& L, int64_t rb, int64_t c0) {
    if (c0 >= L.da) return;
    float v[COLS][32];
    const int rows = (int)min<int64_t>(32, L.rows - rb * 32);
    const bool in = c0 < L.cols;     // else the column of ones
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        const int64_t at = (rb * 32 + min(r, rows - 1)) * L.cols + (in ? c0 : 0);
        if constexpr (COLS == 2) {
            const uint32_t u = as_global(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(L.x) + at))[0];
            v[0][r] = __uint_as_float(u << 16);
            v[1][r] = __uint_as_float(u & 0xffff0000u);
        } else if constexpr (BF16) {
            v[0][r] = bf16_to_f32(as_global(static_cast<const uint16_t*>(L.x))[at]);
        } else {
            v[0][r] = as_global(static_cast<const float*>(L.x))[at];
        }
    }
#pragma unroll
    for (int r = 0; r < 32; ++r)
#pragma unroll
        for (int c = 0; c < COLS; ++c) v[c][r] = r >= rows ? 0.0f : in ? v[c][r] : 1.0f;
    const int64_t at = rb * L.da + c0;
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        if (c > 0 && c0 + c >= L.da) break;   // the column of ones stands alone
        uint4v code[2];
        uint8_t s;
        encode(v[c], code, s);
        uint4v* p = reinterpret_cast<uint4v*>(L.codes + (at + c) * 32);
        as_global(p)[0] = code[0];
        as_global(p)[1] = code[1];
        as_global(L.scales)[at + c] = s;
    }
}

template <bool BF16>
__global__ __launch_bounds__(NT) void keep_store_kernel(KeepLaunch P) {
    const KeepLayer& L = P.layer[find_layer(P, blockIdx.x)];
    const int64_t t = blockIdx.x - L.block_begin;
    const int64_t rb = t / L.groups, c = (t % L.groups) * NT + threadIdx.x;
    if constexpr (BF16) {
        if (L.pair) {
            store_block<BF16, 2>(L, rb, 2 * c);
            return;
        }
    }
    store_block<BF16, 1>(L, rb, c);
}

// Two codes (byte pair `hi` of w) times s as bfloat16, exact.
__device__ __forceinline__ bf16x2 decode2(uint32_t w, float s, bool hi) {
    return hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, s, true)
              : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, s, false);
}

template <bool BF16, int COLS>
__device__ __forceinline__ void load_block(const KeepLayer& L, int64_t rb, int64_t c0) {
    if (c0 >= L.cols) return;
    bf16x2 v[COLS][16];
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        const int64_t at = rb * L.da + c0 + c;
        const float s = __uint_as_float((uint32_t)as_global(L.scales)[at] << 23);
        const uint4v* p = reinterpret_cast<const uint4v*>(L.codes + at * 32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4v q = as_global(p)[h];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                v[c][8 * h + 2 * w] = decode2(q[w], s, false);
                v[c][8 * h + 2 * w + 1] = decode2(q[w], s, true);
            }
        }
    }
    const int rows = (int)min<int64_t>(32, L.rows - rb * 32);
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        if (r >= rows) break;
        const int64_t at = (rb * 32 + r) * L.cols + c0;
        if constexpr (COLS == 2) {
            const bf16x2 u = {v[0][r >> 1][r & 1], v[1][r >> 1][r & 1]};
            *as_global(reinterpret_cast<bf16x2*>(static_cast<__bf16*>(L.x) + at)) = u;
        } else if constexpr (BF16) {
            as_global(static_cast<__bf16*>(L.x))[at] = v[0][r >> 1][r & 1];
        } else {
            as_global(static_cast<float*>(L.x))[at] = (float)v[0][r >> 1][r & 1];
        }
    }
}

template <bool BF16>
__global__ __launch_bounds__(NT) void keep_load_kernel(KeepLaunch P) {
    const KeepLayer& L = P.layer[find_layer(P, blockIdx.x)];
    const int64_t t = blockIdx.x - L.block_begin;
    const int64_t rb = t / L.groups, c = (t % L.groups) * NT + threadIdx.x;
    if constexpr (BF16) {
        if (L.pair) {
            load_block<BF16, 2>(L, rb, 2 * c);
            return;
        }
    }
    load_block<BF16, 1>(L, rb, c);
}

// --------------------------------------------------------------- products --

// 128 columns of two blocks of codes in LDS: 32 bytes per column and block,
// the halves of columns 8 .. 15 of every 16 exchanged, so that 16 lanes
// reading one half of 16 columns fall on different banks.
struct CodeSlab {
    static constexpr int BYTES = 2 * kKeepTile * 32;
    static constexpr int COPIES = BYTES / 16 / NT;   // 2 per thread, one per block
    static __device__ __forceinline__ int at(int block, int col, int half) {
        return block * (kKeepTile * 32) + col * 32 + ((half ^ ((col >> 3) & 1)) << 4);
    }
    // columns from col0 on of blocks rb and rb + 1; zero from column `da`
    // and block `end` on
    static __device__ __forceinline__ void load(uint4v (&r)[COPIES], const uint8_t* codes, int64_t rb, int end,
                                                int col0, int da) {
        const int col = threadIdx.x >> 1, half = threadIdx.x & 1;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(codes + (rb * da + col0) * 32), (short)0, 0x7fffffff, 0x00020000);
#pragma unroll
        for (int k = 0; k < COPIES; ++k) {
            const uint32_t off =
                (col0 + col < da && rb + k < end) ? (uint32_t)(k * da * 32 + col * 32 + half * 16) : kOOB;
            r[k] = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
        }
    }
    static __device__ __forceinline__ void store(char* lds, const uint4v (&r)[COPIES]) {
        const int col = threadIdx.x >> 1, half = threadIdx.x & 1;
#pragma unroll
        for (int k = 0; k < COPIES; ++k) *reinterpret_cast<uint4v*>(lds + at(k, col, half)) = r[k];
    }
};

// Scale byte of block rb and column `col` (1.0 for what lies outside: the codes there are zero).
__device__ __forceinline__ int scale_of(const uint8_t* scales, int64_t rb, int end, int col, int da) {
    const bool ok = rb < end && col < da;
    const int s = as_global(scales)[ok ? rb * da + col : 0];
    return ok ? s : 127;
}

__device__ __forceinline__ int find_prob(const KeepProbs& L, int64_t item, int64_t KeepProb::*begin) {
    int k = 0;
    while (k + 1 < L.n && L.p[k + 1].*begin <= item) ++k;
    return k;
}

__device__ __forceinline__ void keep_out(const KeepProbs& L, const KeepProb& P, bool factor, int i, int j, float v) {
    if (i >= P.m || j >= P.da || (factor && j < i)) return;
    float* p = P.out + (int64_t)i * P.da + j;
    if (factor) {
        v *= P.alpha;
        if (!L.first_step) v = L.eps * *as_global(p) + (1.0f - L.eps) * v;
    }
    *as_global(p) = v;
}

// A finished tile: to its partial buffer where the rows are split, else out.
__device__ __forceinline__ void keep_tile_out(const KeepProbs& L, const KeepProb& P, bool factor,
                                              const floatx16 (&acc)[2][2], int kc, int t, int m0, int n0, int wm, int wn,
                                              int lane) {
    const int g = lane >> 5;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int i = 64 * wm + 32 * a + 8 * (r >> 2) + 4 * g + (r & 3), j = 64 * wn + 32 * b + (lane & 31);
                if (P.ksplit > 1)
                    as_global(P.part)[((int64_t)kc * P.ntiles + t) * (kKeepTile * kKeepTile) + i * kKeepTile + j] =
                        acc[a][b][r];
                else
                    keep_out(L, P, factor, m0 + i, n0 + j, acc[a][b][r]);
            }
}

// The 16 codes of rows 16 g .. 16 g + 15 (g = lane / 32) of column `col` in
// block `u` of a slab, times their scale: the operands of two products (rows
// 16 g .. + 7 and 16 g + 8 .. + 15; both operands of a product take the rows
// in this order).
__device__ __forceinline__ void code_frags(bf16x8 (&f)[2], const char* slab, int u, int col, int scale, int g) {
    const uint4v c = *reinterpret_cast<const uint4v*>(slab + CodeSlab::at(u, col, g));
    const float s = __uint_as_float((uint32_t)scale << 23);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        union {
            bf16x8 f;
            bf16x2 p[4];
        } v;
#pragma unroll
        for (int w = 0; w < 4; ++w) v.p[w] = decode2(c[2 * h + (w >> 1)], s, w & 1);
        f[h] = v.f;
    }
}

// Factor: upper tiles, two blocks (64 rows) per step.  The block-scaled
// matrix cores would take the codes as they are at twice the rate, but their
// sums keep only about 16 bits of the largest term (an entry of five rows
// came out 3e-5 off); the bf16 ones add exact products in float32.
__global__ __launch_bounds__(NT, 2) void keep_factor_kernel(KeepProbs L) {
    __shared__ __attribute__((aligned(16))) char As[2][CodeSlab::BYTES];
    __shared__ __attribute__((aligned(16))) char Bs[2][CodeSlab::BYTES];
    const int64_t item = xcd_remap(blockIdx.x, gridDim.x);
    const KeepProb& P = L.p[find_prob(L, item, &KeepProb::item_begin)];
    const int64_t q = item - P.item_begin;
    const int kc = (int)(q / P.ntiles), t = (int)(q % P.ntiles);
    int ti, tj;
    upper_band_decode(t, P.tiles_n, 4, ti, tj);
    const int m0 = ti * kKeepTile, n0 = tj * kKeepTile;
    const bool same = ti == tj;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1, g = lane >> 5, col = lane & 31;
    const int begin = kc * P.kchunk, end = min(P.blocks, begin + P.kchunk);
    const bool active = !(same && wm > wn);   // that wave's quarter lies below the diagonal

    floatx16 acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;
    uint4v ra[CodeSlab::COPIES], rb[CodeSlab::COPIES];
    auto fetch = [&](int k) {
        CodeSlab::load(ra, P.codes, k, end, m0, P.da);
        if (!same) CodeSlab::load(rb, P.codes, k, end, n0, P.da);
    };
    auto put = [&](int buf) {
        CodeSlab::store(As[buf], ra);
        if (!same) CodeSlab::store(Bs[buf], rb);
    };
    if (begin < end) {
        fetch(begin);
        put(0);
    }
    __syncthreads();
    int buf = 0;
    for (int k = begin; k < end; k += 2, buf ^= 1) {
        int sa[2][2], sb[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                sa[u][a] = scale_of(P.scales, k + u, end, m0 + 64 * wm + 32 * a + col, P.da);
                sb[u][a] = scale_of(P.scales, k + u, end, n0 + 64 * wn + 32 * a + col, P.da);
            }
        if (k + 2 < end) fetch(k + 2);
        if (active) {
            const char *A = As[buf], *B = same ? As[buf] : Bs[buf];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                bf16x8 fa[2][2], fb[2][2];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    code_frags(fa[a], A, u, 64 * wm + 32 * a + col, sa[u][a], g);
                    code_frags(fb[a], B, u, 64 * wn + 32 * a + col, sb[u][a], g);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[a][h], fb[b][h], acc[a][b], 0, 0, 0);
            }
        }
        if (k + 2 < end) put(buf ^ 1);
        __syncthreads();
    }
    if (active || P.ksplit > 1) keep_tile_out(L, P, true, acc, kc, t, m0, n0, wm, wn, lane);
}

// 128 columns of 32 rows of g in LDS as [row][column] bf16 planes (one, or
// the three parts of float32 values), 256 bytes per row, read with
// transposing reads; the 16-byte chunks of a row are permuted as the rows'
// low bits ask, so that four consecutive rows fall on different banks.
template <bool BF16>
struct GradSlab {
    static constexpr int PLANES = BF16 ? 1 : 3;
    static constexpr int PLANE = kKeepBlock * kKeepTile * 2;
    static constexpr int BYTES = PLANES * PLANE;
    static __device__ __forceinline__ int at(int row, int chunk) {
        return row * 256 + ((chunk ^ (((row & 3) << 2) | ((row >> 2) & 3))) << 4);
    }
    // thread t holds rows t / 16 and t / 16 + 16, columns 8 (t % 16) .. + 7
    using Raw = typename std::conditional<BF16, uint4v[2], uint4v[2][2]>::type;
    static __device__ __forceinline__ void load(Raw& r, const void* g, int64_t row0, int64_t rows, int col0, int m,
                                                bool vec) {
        constexpr int ES = BF16 ? 2 : 4;
        const int c = col0 + 8 * (threadIdx.x & 15);
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(static_cast<const char*>(g) + row0 * m * ES), (short)0, 0x7fffffff, 0x00020000);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = (threadIdx.x >> 4) + 16 * k;
            const bool ok = row0 + row < rows;
            const uint32_t off = (uint32_t)(row * m + c) * ES;
            if (vec) {
                // m is a multiple of 16 bytes: a chunk is inside or wholly past the row
                if constexpr (BF16) {
                    r[k] = __builtin_amdgcn_raw_buffer_load_b128(rs, ok && c < m ? off : kOOB, 0, 0);
                } else {
                    r[k][0] = __builtin_amdgcn_raw_buffer_load_b128(rs, ok && c < m ? off : kOOB, 0, 0);
                    r[k][1] = __builtin_amdgcn_raw_buffer_load_b128(rs, ok && c + 4 < m ? off + 16 : kOOB, 0, 0);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t o = ok && c + e < m ? off + e * ES : kOOB;
                    if constexpr (BF16) {
                        const uint32_t v = __builtin_amdgcn_raw_buffer_load_b16(rs, o, 0, 0);
                        if (e & 1) r[k][e >> 1] |= v << 16;
                        else r[k][e >> 1] = v;
                    } else {
                        r[k][e >> 2][e & 3] = __builtin_amdgcn_raw_buffer_load_b32(rs, o, 0, 0);
                    }
                }
            }
        }
    }
    static __device__ __forceinline__ void store(char* lds, const Raw& r) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = (threadIdx.x >> 4) + 16 * k, chunk = threadIdx.x & 15;
            if constexpr (BF16) {
                *reinterpret_cast<uint4v*>(lds + at(row, chunk)) = r[k];
            } else {
                // x = x0 + x1 + x2, each part the rest rounded to bfloat16 (the last rest has 8 bits)
                uint4v p[3];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    floatx2 x = {__uint_as_float(r[k][e >> 1][2 * (e & 1)]),
                                 __uint_as_float(r[k][e >> 1][2 * (e & 1) + 1])};
#pragma unroll
                    for (int n = 0; n < 3; ++n) {
                        const uint32_t u = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
                        p[n][e] = u;
                        x[0] -= __uint_as_float(u << 16);
                        x[1] -= __uint_as_float(u & 0xffff0000u);
                    }
                }
#pragma unroll
                for (int n = 0; n < 3; ++n) *reinterpret_cast<uint4v*>(lds + n * PLANE + at(row, chunk)) = p[n];
            }
        }
    }
    // columns col0 + lane % 32, rows 16 g + 8 s .. + 7 (g = lane / 32)
    static __device__ __forceinline__ bf16x8 frag(const char* plane, int col0, int s, int lane) {
        const int gr = lane >> 4, p = lane & 15;
        const int col = col0 + 16 * (gr & 1) + 4 * (p & 3), row = 16 * (gr >> 1) + 8 * s + (p >> 2);
        auto rd = [&](int r) {
            const char* a = plane + at(r, col >> 3) + (col & 7) * 2;
            return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) short4v*)const_cast<char*>(a));
        };
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(rd(row), rd(row + 4), 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// Gradient: out[m][da] = g^T x, two blocks (64 rows) per step.  Lane half g
// takes rows 16 g .. 16 g + 15 of a block of codes (one 16-byte read, eight
// conversions), and the columns of g are read in the same row order.
template <bool BF16>
__global__ __launch_bounds__(NT, 2) void keep_grad_kernel(KeepProbs L) {
    using G = GradSlab<BF16>;
    __shared__ __attribute__((aligned(16))) char Gs[2][2 * G::BYTES];
    __shared__ __attribute__((aligned(16))) char Xs[2][CodeSlab::BYTES];
    const int64_t item = xcd_remap(blockIdx.x, gridDim.x);
    const KeepProb& P = L.p[find_prob(L, item, &KeepProb::item_begin)];
    const int64_t q = item - P.item_begin;
    const int kc = (int)(q / P.ntiles), t = (int)(q % P.ntiles);
    const int m0 = (t % P.tiles_m) * kKeepTile, n0 = (t / P.tiles_m) * kKeepTile;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1, half = lane >> 5, col = lane & 31;
    const int begin = kc * P.kchunk, end = min(P.blocks, begin + P.kchunk);

    floatx16 acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;
    uint4v rx[CodeSlab::COPIES];
    typename G::Raw rg[2];
    auto fetch = [&](int k) {
        CodeSlab::load(rx, P.codes, k, end, n0, P.da);
        const int64_t rows = min<int64_t>(P.rows, (int64_t)end * kKeepBlock);
#pragma unroll
        for (int u = 0; u < 2; ++u) G::load(rg[u], P.g, (int64_t)(k + u) * kKeepBlock, rows, m0, P.m, P.vec);
    };
    auto put = [&](int buf) {
        CodeSlab::store(Xs[buf], rx);
#pragma unroll
        for (int u = 0; u < 2; ++u) G::store(Gs[buf] + u * G::BYTES, rg[u]);
    };
    if (begin < end) {
        fetch(begin);
        put(0);
    }
    __syncthreads();
    int buf = 0;
    for (int k = begin; k < end; k += 2, buf ^= 1) {
        int sx[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int b = 0; b < 2; ++b) sx[u][b] = scale_of(P.scales, k + u, end, n0 + 64 * wn + 32 * b + col, P.da);
        if (k + 2 < end) fetch(k + 2);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            bf16x8 fx[2][2];
#pragma unroll
            for (int b = 0; b < 2; ++b) code_frags(fx[b], Xs[buf], u, 64 * wn + 32 * b + col, sx[u][b], half);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = G::PLANES - 1; n >= 0; --n)
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const bf16x8 fg = G::frag(Gs[buf] + u * G::BYTES + n * G::PLANE, 64 * wm + 32 * a, h, lane);
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fg, fx[b][h], acc[a][b], 0, 0, 0);
                    }
        }
        if (k + 2 < end) put(buf ^ 1);
        __syncthreads();
    }
    keep_tile_out(L, P, false, acc, kc, t, m0, n0, wm, wn, lane);
}

// Sums the partial tiles of a split product in chunk order.  Four workgroups
// per tile, 32 rows each.
template <bool FACTOR>
__global__ __launch_bounds__(NT) void keep_reduce_kernel(KeepProbs L) {
    const int64_t tile = blockIdx.x >> 2;
    const KeepProb& P = L.p[find_prob(L, tile, &KeepProb::red_begin)];
    if (P.ksplit == 1) return;
    const int t = (int)(tile - P.red_begin);
    int ti, tj;
    if constexpr (FACTOR) {
        upper_band_decode(t, P.tiles_n, 4, ti, tj);
    } else {
        ti = t % P.tiles_m;
        tj = t / P.tiles_m;
    }
    const int64_t size = (int64_t)P.ntiles * (kKeepTile * kKeepTile);
    const int j = threadIdx.x & 127;
#pragma unroll 4
    for (int r = 0; r < 16; ++r) {
        const int i = 32 * (int)(blockIdx.x & 3) + 2 * r + (threadIdx.x >> 7);
        const float* p = P.part + (int64_t)t * (kKeepTile * kKeepTile) + i * kKeepTile + j;
        float s = 0.0f;
        for (int k = 0; k < P.ksplit; ++k) s += as_global(p)[k * size];
        keep_out(L, P, FACTOR, ti * kKeepTile + i, tj * kKeepTile + j, s);
    }
}

}  // namespace

hipError_t launch_keep_store(const KeepLaunch& l, int64_t blocks, bool bf16, hipStream_t stream) {
    if (bf16) hipLaunchKernelGGL(keep_store_kernel<true>, dim3((unsigned)blocks), dim3(NT), 0, stream, l);
    else hipLaunchKernelGGL(keep_store_kernel<false>, dim3((unsigned)blocks), dim3(NT), 0, stream, l);
    return hipGetLastError();
}

hipError_t launch_keep_load(const KeepLaunch& l, int64_t blocks, bool bf16, hipStream_t stream) {
    if (bf16) hipLaunchKernelGGL(keep_load_kernel<true>, dim3((unsigned)blocks), dim3(NT), 0, stream, l);
    else hipLaunchKernelGGL(keep_load_kernel<false>, dim3((unsigned)blocks), dim3(NT), 0, stream, l);
    return hipGetLastError();
}

hipError_t launch_keep_factor(const KeepProbs& l, int64_t items, hipStream_t stream) {
    hipLaunchKernelGGL(keep_factor_kernel, dim3((unsigned)items), dim3(NT), 0, stream, l);
    return hipGetLastError();
}

hipError_t launch_keep_grad(const KeepProbs& l, int64_t items, bool bf16, hipStream_t stream) {
    if (bf16) hipLaunchKernelGGL(keep_grad_kernel<true>, dim3((unsigned)items), dim3(NT), 0, stream, l);
    else hipLaunchKernelGGL(keep_grad_kernel<false>, dim3((unsigned)items), dim3(NT), 0, stream, l);
    return hipGetLastError();
}

hipError_t launch_keep_reduce(const KeepProbs& l, int64_t tiles, bool factor, hipStream_t stream) {
    if (tiles == 0) return hipSuccess;
    const dim3 grid((unsigned)(4 * tiles));
    if (factor) hipLaunchKernelGGL(keep_reduce_kernel<true>, grid, dim3(NT), 0, stream, l);
    else hipLaunchKernelGGL(keep_reduce_kernel<false>, grid, dim3(NT), 0, stream, l);
    return hipGetLastError();
}

}  // namespace kfac
