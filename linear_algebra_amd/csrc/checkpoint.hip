// Layer inputs kept in 8 bits between the forward and the backward pass, and
// the two products that use them: the factor A = x^T x / rows and the
// gradient [dW | db] = g^T [x | 1].
//
// Both products sum over rows, so a block shares its scale along the rows of
// one column: 32 consecutive rows, e4m3 codes and one power of two, next to
// one another in memory as the matrix cores take them.  A code times its
// power of two is exactly a bfloat16 number (4 significant bits), so the
// codes are converted on the way to the bf16 matrix cores without a rounding;
// float32 gradients enter as three bf16 parts, exact from 2^-103 on.
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
    for (int i = 1; i < L.n; ++i)
        if (L.layer[i].block_begin <= block) k = i;
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

// Two neighbouring bf16 elements as one access; rows of odd width start on
// 2-byte boundaries, which the global accesses of this part allow.
struct __attribute__((packed, aligned(2))) Pair {
    uint32_t v;
};

// Workgroups take runs of columns of one block of rows, one column of
// float32 or two of bf16 per thread: a wave reads 256 bytes of each of the
// 32 rows and writes the columns' codes, 32 bytes each, next to one another.
// The values stay in registers between the maximum and the conversion, so
// each is read once.  The code is rounded to nearest even, 2^-4 of a value at
// most: what keeping a quarter of float32's or half of bfloat16's bytes costs.
// 4096 x 4097 bfloat16: 51 MB in 15.5 us, 3.3 TB/s (kfac_stream_copy: 6.1);
// 128 x 1025 float32: 3.4 us, a launch.
template <bool BF16>
__global__ __launch_bounds__(NT) void keep_store_kernel(KeepLaunch P) {
    constexpr int COLS = BF16 ? 2 : 1;
    const KeepLayer& L = P.layer[find_layer(P, blockIdx.x)];
    const uint32_t t = blockIdx.x - (uint32_t)L.block_begin;
    const int64_t rb = t / (uint32_t)L.groups;
    const int c0 = (int)((t % (uint32_t)L.groups) * NT + threadIdx.x) * COLS;
    const int da = L.da, cols = L.cols;
    if (c0 >= da) return;
    float v[COLS][32];
    const int rows = (int)min<int64_t>(32, L.rows - rb * 32);
    const int64_t first = rb * 32 * cols + min(c0, cols - 1);
    if constexpr (BF16) {
        const uint16_t* x = static_cast<const uint16_t*>(L.x) + first;
        if (c0 + 1 < cols) {
#pragma unroll
            for (int r = 0; r < 32; ++r) {
                const uint32_t u = as_global(reinterpret_cast<const Pair*>(x + (int64_t)min(r, rows - 1) * cols))->v;
                v[0][r] = __uint_as_float(u << 16);
                v[1][r] = __uint_as_float(u & 0xffff0000u);
            }
        } else {
            // the last column, or the column of ones
#pragma unroll
            for (int r = 0; r < 32; ++r) {
                v[0][r] = bf16_to_f32(as_global(x)[(int64_t)min(r, rows - 1) * cols]);
                v[1][r] = 1.0f;
            }
        }
    } else {
        const float* x = static_cast<const float*>(L.x) + first;
#pragma unroll
        for (int r = 0; r < 32; ++r) v[0][r] = as_global(x)[(int64_t)min(r, rows - 1) * cols];
    }
    const bool in = c0 < cols;
#pragma unroll
    for (int r = 0; r < 32; ++r)
#pragma unroll
        for (int c = 0; c < COLS; ++c) v[c][r] = r >= rows ? 0.0f : in ? v[c][r] : 1.0f;
    const int64_t at = rb * da + c0;
    uint8_t* scales = L.scales;
    uint8_t* codes = L.codes;
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        if (c > 0 && c0 + c >= da) break;
        uint4v code[2];
        uint8_t s;
        encode(v[c], code, s);
        uint4v* p = reinterpret_cast<uint4v*>(codes + (at + c) * 32);
        as_global(p)[0] = code[0];
        as_global(p)[1] = code[1];
        as_global(scales)[at + c] = s;
    }
}

// Two codes (byte pair `hi` of w) times s as bfloat16, exact.
__device__ __forceinline__ bf16x2 decode2(uint32_t w, float s, bool hi) {
    return hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, s, true)
              : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, s, false);
}

// Half a block (16 rows) per thread, columns as in the store.  4096 x 4097 to
// bfloat16: 51 MB in 12.5 us, 4.1 TB/s.
template <bool BF16>
__global__ __launch_bounds__(NT) void keep_load_kernel(KeepLaunch P) {
    constexpr int COLS = BF16 ? 2 : 1;
    const KeepLayer& L = P.layer[find_layer(P, blockIdx.x)];
    const uint32_t t = blockIdx.x - (uint32_t)L.block_begin;
    const int64_t r16 = t / (uint32_t)L.groups;
    const int c0 = (int)((t % (uint32_t)L.groups) * NT + threadIdx.x) * COLS;
    const int cols = L.cols;
    const int rows = (int)min<int64_t>(16, L.rows - r16 * 16);
    if (c0 >= cols) return;
    uint32_t v[COLS][8];     // rows 2 w (low half) and 2 w + 1
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        const int64_t at = (r16 >> 1) * L.da + min(c0 + c, cols - 1);
        const float s = __uint_as_float((uint32_t)as_global(L.scales)[at] << 23);
        const uint4v q = *as_global(reinterpret_cast<const uint4v*>(L.codes + at * 32 + (r16 & 1) * 16));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            v[c][2 * w] = __builtin_bit_cast(uint32_t, decode2(q[w], s, false));
            v[c][2 * w + 1] = __builtin_bit_cast(uint32_t, decode2(q[w], s, true));
        }
    }
    const int64_t first = r16 * 16 * cols + c0;
    const bool two = COLS == 2 && c0 + 1 < cols;
    auto rows_out = [&](auto pair, auto full) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (!decltype(full)::value && r >= rows) return;
            const uint32_t x = v[0][r >> 1], y = v[COLS - 1][r >> 1];
            if constexpr (!BF16) {
                as_global(static_cast<float*>(L.x))[first + (int64_t)r * cols] =
                    __uint_as_float(r & 1 ? x & 0xffff0000u : x << 16);
            } else if constexpr (decltype(pair)::value) {
                as_global(reinterpret_cast<Pair*>(static_cast<uint16_t*>(L.x) + first + (int64_t)r * cols))->v =
                    r & 1 ? (x >> 16) | (y & 0xffff0000u) : (x & 0xffffu) | (y << 16);
            } else {
                as_global(static_cast<uint16_t*>(L.x))[first + (int64_t)r * cols] = (uint16_t)(r & 1 ? x >> 16 : x);
            }
        }
    };
    if (rows == 16) {
        if (two) rows_out(std::true_type(), std::true_type());
        else rows_out(std::false_type(), std::true_type());
    } else {
        if (two) rows_out(std::true_type(), std::false_type());
        else rows_out(std::false_type(), std::false_type());
    }
}

// --------------------------------------------------------------- products --

// 128 columns of two blocks of codes in LDS: 32 bytes per column and block,
// the halves of columns 8 .. 15 of every 16 exchanged, so that 16 lanes
// reading one half of 16 columns fall on different banks; then the scales as
// float32 (one byte load and one conversion per thread and pair of blocks).
struct CodeSlab {
    static constexpr int CODES = 2 * kKeepTile * 32;
    static constexpr int BYTES = CODES + 2 * kKeepTile * 4;
    static constexpr int PIECES = 3;     // a thread's accesses per slab: one per block, and a scale
    struct Raw {
        uint4v c[2];
        uint32_t s;
    };
    // where the next slab begins, and blocks left from there
    const uint8_t *codes, *scales;
    int left, da, col0;
    uint32_t off[2], soff;               // this thread's 16 bytes of either block, and its scale
    int put_at, tid;                     // tid: 0 .. 255 among the threads that fill the slab
    __amdgpu_buffer_rsrc_t rc, rs;       // the slab being fetched

    static __device__ __forceinline__ int at(int block, int col, int half) {
        return block * (kKeepTile * 32) + col * 32 + ((half ^ ((col >> 3) & 1)) << 4);
    }
    // columns from `first` on, blocks [begin, end); what lies past them reads as zero
    __device__ __forceinline__ CodeSlab(const KeepProb& P, int first, int begin, int end, int thread)
        : codes(P.codes + ((int64_t)begin * P.da + first) * 32), scales(P.scales + (int64_t)begin * P.da + first),
          left(end - begin), da(P.da), col0(first), tid(thread) {
        const int col = tid >> 1, half = tid & 1;
        const int sk = tid >> 7, sc = tid & (kKeepTile - 1);
        off[0] = first + col < da ? (uint32_t)(col * 32 + half * 16) : kOOB;
        off[1] = first + col < da ? off[0] + (uint32_t)da * 32 : kOOB;
        soff = first + sc < da ? (uint32_t)(sk * da + sc) : kOOB;
        put_at = at(0, col, half);
    }
    // on to the next two blocks (their ranges end with the last block)
    __device__ __forceinline__ void next() {
        const int n = max(0, min(2, left) * da - col0);
        rc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(codes), (short)0, n * 32, 0x00020000);
        rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(scales), (short)0, n, 0x00020000);
        codes += 64 * (int64_t)da;
        scales += 2 * da;
        left -= 2;
    }
    __device__ __forceinline__ void load(Raw& r, int p) const {
        if (p < 2) r.c[p] = __builtin_amdgcn_raw_buffer_load_b128(rc, off[p], 0, 0);
        else r.s = __builtin_amdgcn_raw_buffer_load_b8(rs, soff, 0, 0);
    }
    __device__ __forceinline__ void put(char* lds, const Raw& r, int p) const {
        if (p < 2) *reinterpret_cast<uint4v*>(lds + p * (kKeepTile * 32) + put_at) = r.c[p];
        else reinterpret_cast<uint32_t*>(lds + CODES)[tid] = r.s << 23;
    }
    // The 16 codes of rows 16 g .. 16 g + 15 of column `col` in block `u`,
    // and their scale: the operands of two products (half 0: rows 16 g ..
    // + 7, half 1: 16 g + 8 .. + 15; both operands of a product take the
    // rows in this order).
    struct Codes {
        uint4v c;
        float s;
        __device__ __forceinline__ void read(const char* lds, int u, int col, int g) {
            c = *reinterpret_cast<const uint4v*>(lds + at(u, col, g));
            s = reinterpret_cast<const float*>(lds + CODES)[u * kKeepTile + col];
        }
        __device__ __forceinline__ bf16x8 operand(int half) const {
            union {
                bf16x8 f;
                bf16x2 p[4];
            } v;
#pragma unroll
            for (int w = 0; w < 4; ++w) v.p[w] = decode2(c[2 * half + (w >> 1)], s, w & 1);
            return v.f;
        }
    };
};

// Neighbouring items to one XCD, the whole tiles and the chunks each shared
// out evenly (together, some XCDs would get chunks only).
__device__ __forceinline__ int64_t keep_item(const KeepProbs& L) {
    const int64_t b = blockIdx.x;
    return b < L.cut ? xcd_remap(b, L.cut) : L.cut + xcd_remap(b - L.cut, gridDim.x - L.cut);
}

// Work item of a product launch: tiles [0, whole) take all rows in one item,
// the others are split in `ksplit` chunks.
struct KeepWork {
    int t, kc, begin, end;
    bool split;
    __device__ __forceinline__ KeepWork(const KeepProb& P, uint32_t q) {
        split = q >= (uint32_t)P.whole;
        if (split) {
            q -= P.whole;
            const uint32_t rest = P.ntiles - P.whole;
            kc = (int)(q / rest);
            t = (int)(q % rest) + P.whole;
            begin = kc * P.kchunk;
            end = min(P.blocks, begin + P.kchunk);
        } else {
            t = (int)q;
            kc = 0;
            begin = 0;
            end = P.blocks;
        }
    }
};

__device__ __forceinline__ int find_prob(const KeepProbs& L, int64_t item, int64_t KeepProb::*begin) {
    int k = 0;
    for (int i = 1; i < L.n; ++i)
        if (L.p[i].*begin <= item) k = i;
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
// Tiles that lie wholly inside (and above the diagonal) are written without
// a test per element.
// `a`: which 32 rows of the wave's 64.
template <bool FACTOR>
__device__ __forceinline__ void keep_rows_out(const KeepProbs& L, const KeepProb& P, const KeepWork& W,
                                              const floatx16 (&acc)[2], int a, int m0, int n0, int wm, int wn, int lane) {
    const int g = lane >> 5;
    const bool inside = m0 + kKeepTile <= P.m && n0 + kKeepTile <= P.da && !(FACTOR && m0 == n0);
    // (row, column) of the wave's first element for each block and register, the lane's own offset apart
    auto each = [&](auto f) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) f(acc[b][r], 64 * wm + 32 * a + 8 * (r >> 2) + (r & 3), 64 * wn + 32 * b);
    };
    if (W.split) {
        float* part = P.part + ((int64_t)W.kc * (P.ntiles - P.whole) + (W.t - P.whole)) * (kKeepTile * kKeepTile);
        const int own = 4 * g * kKeepTile + (lane & 31);
        each([&](float v, int i, int j) { as_global(part + i * kKeepTile + j)[own] = v; });
    } else if (inside) {
        float* out = P.out + (int64_t)m0 * P.da + n0;
        const int own = 4 * g * P.da + (lane & 31);
        if (!FACTOR) {
            each([&](float v, int i, int j) { as_global(out + (int64_t)i * P.da + j)[own] = v; });
        } else if (L.first_step) {
            each([&](float v, int i, int j) { as_global(out + (int64_t)i * P.da + j)[own] = v * P.alpha; });
        } else {
            each([&](float v, int i, int j) {
                auto* p = &as_global(out + (int64_t)i * P.da + j)[own];
                *p = L.eps * *p + (1.0f - L.eps) * (v * P.alpha);
            });
        }
    } else {
        each([&](float v, int i, int j) { keep_out(L, P, FACTOR, m0 + i + 4 * g, n0 + j + (lane & 31), v); });
    }
}

// Order of a product group for the scheduler: its LDS reads (the next group's
// operands), then N products, each with other instructions in its shadow: V
// vector ones, a global load and an LDS write.
template <int N, int V>
__device__ __forceinline__ void shadow() {
    __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// The steps of a work item, two blocks of 32 rows each.  The products of a
// step read one LDS buffer; beside them, piece by piece, the next step's
// data goes from registers to the other buffer and the data of the step
// after it is fetched.  (Issued in one go between the products, loads and
// writes took as long as they did.)  Fetches past the end read nothing
// (zeros), and are not branched around: behind a branch, the wait for a
// step's data would also wait for the fetches after it.
template <typename Stage, int PIECES, typename Fetch, typename Put, typename Products>
__device__ __forceinline__ void pipeline(int blocks, Fetch fetch, Put put, Products products) {
    if (blocks <= 0) return;
    Stage even, odd;
#pragma unroll
    for (int p = 0; p < PIECES; ++p) fetch(even, p);
#pragma unroll
    for (int p = 0; p < PIECES; ++p) fetch(odd, p);
#pragma unroll
    for (int p = 0; p < PIECES; ++p) put(even, 0, p);
    __syncthreads();
    for (int k = 0;; k += 4) {
        products(0, [&](int p) { fetch(even, p); }, [&](int p) { put(odd, 1, p); });
        if (k + 2 >= blocks) break;
        __syncthreads();
        products(1, [&](int p) { fetch(odd, p); }, [&](int p) { put(even, 0, p); });
        if (k + 4 >= blocks) break;
        __syncthreads();
    }
}

// Factor: upper tiles, two blocks (64 rows) per step.  The block-scaled
// matrix cores would take the codes as they are at twice the rate, but their
// sums keep only about 16 bits of the largest term (an entry of five rows
// came out 3e-5 off); the bf16 ones add exact products in float32.  4096 rows:
// width 4097 72 us, 955 TFLOP/s of the 1283 of a large library product (561
// tiles of 128 x 128, 33 of them for the last column alone), bound by the
// conversions between the matrix instructions; width 1025 15 to 18 us, a
// single round of 225 chunks, most of it the way to and from the loop.
__global__ __launch_bounds__(NT, 2) void keep_factor_kernel(KeepProbs L) {
    __shared__ __attribute__((aligned(16))) char As[2][CodeSlab::BYTES];
    __shared__ __attribute__((aligned(16))) char Bs[2][CodeSlab::BYTES];
    const int64_t item = keep_item(L);
    const KeepProb& P = L.p[find_prob(L, item, &KeepProb::item_begin)];
    const KeepWork W(P, (uint32_t)(item - P.item_begin));
    int ti, tj;
    upper_band_decode(W.t, P.tiles_n, 4, ti, tj);
    const int m0 = ti * kKeepTile, n0 = tj * kKeepTile;
    const bool same = ti == tj;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1, g = lane >> 5, col = lane & 31;
    // a quarter below the diagonal or past the last column has nothing to
    // add, nor has the right half of one
    const bool active = !(same && wm > wn) && n0 + 64 * wn < P.da;
    const bool both = n0 + 64 * wn + 32 < P.da;

    floatx16 acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;
    CodeSlab sa(P, m0, W.begin, W.end, threadIdx.x), sb(P, n0, W.begin, W.end, threadIdx.x);
    struct Stage {
        CodeSlab::Raw a, b;
    };
    constexpr int PIECES = 2 * CodeSlab::PIECES;
    auto fetch = [&](Stage& r, int p) {
        if (p == 0) {
            sa.next();
            sb.next();
        }
        if (p < CodeSlab::PIECES) sa.load(r.a, p);
        else sb.load(r.b, p - CodeSlab::PIECES);
    };
    auto put = [&](const Stage& r, int buf, int p) {
        if (p < CodeSlab::PIECES) sa.put(As[buf], r.a, p);
        else sb.put(Bs[buf], r.b, p - CodeSlab::PIECES);
    };
    // The operands of product group j + 1 are formed in the shadow of group
    // j's products.
    auto products = [&](const char* A, const char* B, auto blocks, auto fetch1, auto put1) {
        constexpr int NB = decltype(blocks)::value;
        CodeSlab::Codes ca[2][2], cb[2][NB];
        bf16x8 fa[2][2], fb[2][NB];
        auto read = [&](int u) {
#pragma unroll
            for (int a = 0; a < 2; ++a) ca[u][a].read(A, u, 64 * wm + 32 * a + col, g);
#pragma unroll
            for (int b = 0; b < NB; ++b) cb[u][b].read(B, u, 64 * wn + 32 * b + col, g);
        };
        auto form = [&](int j) {
#pragma unroll
            for (int a = 0; a < 2; ++a) fa[j & 1][a] = ca[j >> 1][a].operand(j & 1);
#pragma unroll
            for (int b = 0; b < NB; ++b) fb[j & 1][b] = cb[j >> 1][b].operand(j & 1);
        };
        read(0);
        read(1);
        form(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    acc[a][b] =
                        __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[j & 1][a], fb[j & 1][b], acc[a][b], 0, 0, 0);
            if (j < 3) form(j + 1);
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                if (p * 2 / PIECES == j) fetch1(p);
                if (p * 2 / PIECES + 2 == j) put1(p);
            }
            shadow<2 * NB, 6>();
        }
    };
    if (active && both) {
        pipeline<Stage, PIECES>(W.end - W.begin, fetch, put, [&](int buf, auto fetch1, auto put1) {
            products(As[buf], Bs[buf], std::integral_constant<int, 2>(), fetch1, put1);
        });
    } else {
        pipeline<Stage, PIECES>(W.end - W.begin, fetch, put, [&](int buf, auto fetch1, auto put1) {
#pragma unroll
            for (int p = 0; p < PIECES; ++p) fetch1(p);
#pragma unroll
            for (int p = 0; p < PIECES; ++p) put1(p);
            if (active) products(As[buf], Bs[buf], std::integral_constant<int, 1>(), [](int) {}, [](int) {});
        });
    }
    if (active || W.split) {
#pragma unroll
        for (int a = 0; a < 2; ++a) keep_rows_out<true>(L, P, W, acc[a], a, m0, n0, wm, wn, lane);
    }
}

// 128 columns of 32 rows of g in LDS as [row][column] bf16 planes (one, or
// the three parts of float32 values), 256 bytes per row, read with
// transposing reads; the 16-byte chunks of a row are permuted as the rows'
// low bits ask, so that four consecutive rows fall on different banks.
template <bool BF16, bool WORD>
struct GradSlab {
    static constexpr int PLANES = BF16 ? 1 : 3;
    static constexpr int PLANE = kKeepBlock * kKeepTile * 2;
    static constexpr int BYTES = PLANES * PLANE;
    static __device__ __forceinline__ int at(int row, int chunk) {
        return row * 256 + ((chunk ^ (((row & 3) << 2) | ((row >> 2) & 3))) << 4);
    }
    // thread t holds rows t / 16 + 16 p (piece p), columns 8 (t % 16) .. + 7
    static constexpr int ES = BF16 ? 2 : 4;
    static constexpr int WORDS = BF16 ? 1 : 2;
    static constexpr int PIECES = 4;
    struct Raw {
        uint4v v[PIECES][WORDS];
        uint32_t next[WORD ? 1 : PIECES];   // the word behind
    };
    const char* g;               // where the next 64 rows begin, on a 4-byte boundary
    int64_t left;                // rows left from there
    int m, tid;
    int lead;                    // bytes between that boundary and the rows
    int odd;                     // 16 where this thread's first column is the upper half of its word
    int last;                    // last row of the current 64
    uint32_t off[PIECES][WORDS];
    __amdgpu_buffer_rsrc_t rg;
    // Columns from col0 on, rows [row0, last); the rows past them read as
    // zero.  A thread's columns past the last one are the next row's: they
    // lead to rows of the result that are not written.
    __device__ __forceinline__ GradSlab(const KeepProb& P, int col0, int64_t row0, int64_t last, int thread)
        : left(last - row0), m(P.m), tid(thread) {
        g = static_cast<const char*>(P.g) + row0 * m * ES;
        lead = WORD ? 0 : (int)(reinterpret_cast<uintptr_t>(g) & 2);
        g -= lead;
        const int c = col0 + 8 * (tid & 15);
        odd = WORD ? 0 : (((tid >> 4) * m + lead / 2) & 1) * 16;   // (the same in every piece and step)
#pragma unroll
        for (int p = 0; p < PIECES; ++p)
#pragma unroll
            for (int w = 0; w < WORDS; ++w)
                off[p][w] = m - c > w * 16 / ES
                                ? ((uint32_t)(((tid >> 4) + 16 * p) * m + c) * ES + lead + 16 * w) & ~3u
                                : kOOB;
    }
    __device__ __forceinline__ void next() {
        // (the range ends on a word, in whose lower half the last row may end)
        const int n = (int)max<int64_t>(0, min<int64_t>(64, left));
        last = n - 1;
        rg = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(g), (short)0, n ? (n * m * ES + lead + 3) & ~3 : 0,
                                               0x00020000);
        g += 64 * (int64_t)m * ES;
        left -= 64;
    }
    __device__ __forceinline__ void load(Raw& r, int p) const {
        // the row behind the last may begin in its last word: past the range from there on
        const uint32_t past = WORD ? 0 : (uint32_t)(last - ((tid >> 4) + 16 * p)) & kOOB;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) r.v[p][w] = __builtin_amdgcn_raw_buffer_load_b128(rg, off[p][w] | past, 0, 0);
        if constexpr (!WORD) r.next[p] = __builtin_amdgcn_raw_buffer_load_b32(rg, (off[p][0] | past) + 16, 0, 0);
    }
    __device__ __forceinline__ void put(char* lds, const Raw& r, int p) const {
        const int at0 = (p >> 1) * BYTES + at((tid >> 4) + 16 * (p & 1), tid & 15);
        if constexpr (BF16) {
            uint4v v = r.v[p][0];
            if constexpr (!WORD) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = __builtin_amdgcn_alignbit(e < 3 ? v[e + 1] : r.next[p], v[e], (uint32_t)odd);
            }
            *reinterpret_cast<uint4v*>(lds + at0) = v;
        } else {
            // x = x0 + x1 + x2, each part the upper half of the rest's bits (8
            // of its 24, sign and exponent apart).  Cut, not rounded: a number
            // past bfloat16's largest stays finite.  The rests are those of
            // the nearest finite number: infinity - infinity would turn an
            // infinity into NaN.  (A signalling NaN may come out as an
            // infinity.)  Bits under 2^-133 are cut off, and parts
            // under 2^-126 may come out of the product as zero.
            uint4v q[3];
            const float most = __uint_as_float(0x7f7fffffu);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[2] = {__uint_as_float(r.v[p][e >> 1][2 * (e & 1)]),
                              __uint_as_float(r.v[p][e >> 1][2 * (e & 1) + 1])};
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    // the upper halves of both
                    q[n][e] = __builtin_amdgcn_perm(__float_as_uint(x[1]), __float_as_uint(x[0]), 0x07060302u);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (n == 0) x[k] = __builtin_amdgcn_fmed3f(x[k], -most, most);
                        x[k] -= __uint_as_float(__float_as_uint(x[k]) & 0xffff0000u);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < 3; ++n) *reinterpret_cast<uint4v*>(lds + n * PLANE + at0) = q[n];
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
// TEAMS = 2: two teams of four waves take half of the rows each and add their
// sums through LDS, so that every SIMD holds two waves where there is one
// tile per compute unit (4096 x 1024 x 4097 bfloat16: 47 us, with one team
// 51; 730 TFLOP/s with its 8 tiles of one column, bound by LDS: each step
// reads g by columns and the codes by rows).  float32 gradients keep one team:
// their three parts fill the registers.  128 x 1024 x 2049 in float32: 10.5
// us, four blocks per tile and the way to and from them; 4096 x 1024 x 4097: 123
// us, with parts rounded instead of cut (infinite ones then become NaN) 121.
// WORD: rows of g start on 4-byte boundaries.  bfloat16 rows that do not are
// read by the words they lie in, one more per 16 bytes, and shifted into place
// (4096 x 1023 x 4097: 59 us; rows of 1022, on 4-byte boundaries, 48; read
// element by element 174).
template <bool BF16, bool WORD, int TEAMS>
__global__ __launch_bounds__(NT * TEAMS, TEAMS) void keep_grad_kernel(KeepProbs L) {
    using G = GradSlab<BF16, WORD>;
    __shared__ __attribute__((aligned(16))) char Gall[TEAMS][2][2 * G::BYTES];
    __shared__ __attribute__((aligned(16))) char Xall[TEAMS][2][CodeSlab::BYTES];
    const int64_t item = keep_item(L);
    const KeepProb& P = L.p[find_prob(L, item, &KeepProb::item_begin)];
    const KeepWork W(P, (uint32_t)(item - P.item_begin));
    const int m0 = (W.t % P.tiles_m) * kKeepTile, n0 = (W.t / P.tiles_m) * kKeepTile;
    const int lane = threadIdx.x & 63, all = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int team = all >> 2, wave = all & 3, thread = threadIdx.x & (NT - 1);
    char (&Gs)[2][2 * G::BYTES] = Gall[team];
    char (&Xs)[2][CodeSlab::BYTES] = Xall[team];
    const int wm = wave >> 1, wn = wave & 1, half = lane >> 5, col = lane & 31;
    const bool active = m0 + 64 * wm < P.m && n0 + 64 * wn < P.da;
    const bool both = n0 + 64 * wn + 32 < P.da;

    floatx16 acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;
    // this team's blocks
    const int share = ((W.end - W.begin + TEAMS - 1) / TEAMS + 1) & ~1;
    const int begin = W.begin + team * share, end = min(W.end, begin + share);
    CodeSlab sx(P, n0, begin, end, thread);
    G sg(P, m0, (int64_t)begin * kKeepBlock, min<int64_t>(P.rows, (int64_t)end * kKeepBlock), thread);
    struct Stage {
        CodeSlab::Raw x;
        typename G::Raw g;
    };
    constexpr int PIECES = CodeSlab::PIECES + G::PIECES;
    auto fetch = [&](Stage& r, int p) {
        if (p == 0) {
            sg.next();
            sx.next();
        }
        if (p < G::PIECES) sg.load(r.g, p);
        else sx.load(r.x, p - G::PIECES);
    };
    auto put = [&](const Stage& r, int buf, int p) {
        if (p < G::PIECES) sg.put(Gs[buf], r.g, p);
        else sx.put(Xs[buf], r.x, p - G::PIECES);
    };
    // Product group j: block j / (2 PLANES), half j / PLANES % 2 and plane
    // (the smallest part first); the operands of group j + 1 are read and
    // formed in the shadow of group j's products.
    auto products = [&](const char* Gb, const char* X, auto blocks, auto fetch1, auto put1) {
        constexpr int NB = decltype(blocks)::value, PL = G::PLANES, GROUPS = 4 * PL;
        CodeSlab::Codes cx[2][NB];
        bf16x8 fg[2][2], fx[2][NB];
        auto read_codes = [&](int u) {
#pragma unroll
            for (int b = 0; b < NB; ++b) cx[u][b].read(X, u, 64 * wn + 32 * b + col, half);
        };
        auto read_g = [&](int j) {
            const int u = j / (2 * PL), h = j / PL % 2, n = PL - 1 - j % PL;
#pragma unroll
            for (int a = 0; a < 2; ++a)
                fg[j & 1][a] = G::frag(Gb + u * G::BYTES + n * G::PLANE, 64 * wm + 32 * a, h, lane);
        };
        auto form = [&](int q) {
#pragma unroll
            for (int b = 0; b < NB; ++b) fx[q & 1][b] = cx[q >> 1][b].operand(q & 1);
        };
        read_codes(0);
        read_g(0);
        read_codes(1);
        form(0);
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            const int q = j / PL;
            if (j + 1 < GROUPS) read_g(j + 1);
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    acc[a][b] =
                        __builtin_amdgcn_mfma_f32_32x32x16_bf16(fg[j & 1][a], fx[q & 1][b], acc[a][b], 0, 0, 0);
            if (j % PL == PL - 1 && q < 3) form(q + 1);
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                if (p * (GROUPS / 2) / PIECES == j) fetch1(p);
                if (p * (GROUPS / 2) / PIECES + GROUPS / 2 == j) put1(p);
            }
            shadow<2 * NB, BF16 ? 4 : 8>();
        }
    };
    if (active && both) {
        pipeline<Stage, PIECES>(share, fetch, put, [&](int buf, auto fetch1, auto put1) {
            products(Gs[buf], Xs[buf], std::integral_constant<int, 2>(), fetch1, put1);
        });
    } else {
        pipeline<Stage, PIECES>(share, fetch, put, [&](int buf, auto fetch1, auto put1) {
#pragma unroll
            for (int p = 0; p < PIECES; ++p) fetch1(p);
#pragma unroll
            for (int p = 0; p < PIECES; ++p) put1(p);
            if (active) products(Gs[buf], Xs[buf], std::integral_constant<int, 1>(), [](int) {}, [](int) {});
        });
    }
    if constexpr (TEAMS == 1) {
        if (active || W.split) {
#pragma unroll
            for (int a = 0; a < 2; ++a) keep_rows_out<false>(L, P, W, acc[a], a, m0, n0, wm, wn, lane);
        }
    } else {
        // each team hands over one half of its rows and writes the other
        float* X = reinterpret_cast<float*>(&Gall[0][0][0]);
        static_assert(sizeof(Gall) >= 2 * 4 * 2 * 16 * 64 * sizeof(float), "both teams' halves fit");
        auto exchange = [&](auto own) {
            constexpr int A = decltype(own)::value;
            float* give = X + (A * 4 + wave) * 2048;
            const float* take = X + ((1 - A) * 4 + wave) * 2048;
            __syncthreads();
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) give[(16 * b + r) * 64 + lane] = acc[1 - A][b][r];
            __syncthreads();
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    // the first team's rows first, in both halves
                    const float other = take[(16 * b + r) * 64 + lane];
                    acc[A][b][r] = A == 0 ? acc[A][b][r] + other : other + acc[A][b][r];
                }
            if (active || W.split) keep_rows_out<false>(L, P, W, acc[A], A, m0, n0, wm, wn, lane);
        };
        if (team == 0) exchange(std::integral_constant<int, 0>());
        else exchange(std::integral_constant<int, 1>());
    }
}

// Sums the partial tiles of a split product in chunk order: sixteen
// workgroups per tile, four neighbouring elements per thread.  5 chunks of 45
// tiles: 15 MB in 5 us, as long as the launch takes.
template <bool FACTOR>
__global__ __launch_bounds__(NT) void keep_reduce_kernel(KeepProbs L) {
    const int64_t tile = blockIdx.x >> 4;
    const KeepProb& P = L.p[find_prob(L, tile, &KeepProb::red_begin)];
    const int rest = P.ntiles - P.whole, split = P.ksplit;
    const int u = (int)(tile - P.red_begin), t = u + P.whole;
    int ti, tj;
    if constexpr (FACTOR) {
        upper_band_decode(t, P.tiles_n, 4, ti, tj);
    } else {
        ti = t % P.tiles_m;
        tj = t / P.tiles_m;
    }
    const int e = ((int)(blockIdx.x & 15) * NT + (int)threadIdx.x) * 4;
    const int i = ti * kKeepTile + e / kKeepTile, j = tj * kKeepTile + e % kKeepTile;
    if (i >= P.m || j >= P.da || (FACTOR && j + 3 < i)) return;
    const float* p = P.part + (int64_t)u * (kKeepTile * kKeepTile) + e;
    const int64_t step = (int64_t)rest * (kKeepTile * kKeepTile);
    floatx4 s = *as_global(reinterpret_cast<const floatx4*>(p));
#pragma unroll 8
    for (int k = 1; k < split; ++k) s += *as_global(reinterpret_cast<const floatx4*>(p + k * step));
#pragma unroll
    for (int c = 0; c < 4; ++c) keep_out(L, P, FACTOR, i, j + c, s[c]);
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

hipError_t launch_keep_grad(const KeepProbs& l, int64_t items, bool bf16, bool words, hipStream_t stream) {
    const dim3 grid((unsigned)items);
    // float32 slabs are three times as large: one team's fill the LDS
    if (!bf16) hipLaunchKernelGGL((keep_grad_kernel<false, true, 1>), grid, dim3(NT), 0, stream, l);
    else if (words) hipLaunchKernelGGL((keep_grad_kernel<true, true, 2>), grid, dim3(2 * NT), 0, stream, l);
    else hipLaunchKernelGGL((keep_grad_kernel<true, false, 2>), grid, dim3(2 * NT), 0, stream, l);
    return hipGetLastError();
}

hipError_t launch_keep_reduce(const KeepProbs& l, int64_t tiles, bool factor, hipStream_t stream) {
    if (tiles == 0) return hipSuccess;
    const dim3 grid((unsigned)(16 * tiles));
    if (factor) hipLaunchKernelGGL(keep_reduce_kernel<true>, grid, dim3(NT), 0, stream, l);
    else hipLaunchKernelGGL(keep_reduce_kernel<false>, grid, dim3(NT), 0, stream, l);
    return hipGetLastError();
}

}  // namespace kfac
