// The gated feed-forward block and its backward pass.
//
//   [g | u] = x W^T + b,  h = act(g) u                      (W [2 F][d], gate rows first)
//   dg = dh u act'(g),  du = dh act(g),  dpre = [dg | du]
//   dx = dpre W,  dW = dpre^T x,  db = sum over rows of dpre
//
// The three products run on one kernel of 32 x 32 x 16 matrix-core blocks.
// An operand is read either by rows whose elements are the reduction index
// (x, W forward, dpre for dx) or by rows that are the reduction index itself
// (W for dx; both operands of dW), then with transposing LDS reads.  Slabs of
// BK reduction steps are copied from memory straight into one of two LDS
// buffers while the other is multiplied.  In the forward product a tile's
// columns are F / ... gate columns and the same up columns of W, side by side
// in one wave, so that act(g) u is formed from the accumulators.
//
// float32 operands are split into three bfloat16 parts beforehand (the
// parts add up to the number exactly) and enter as six products, which carry
// a float32 product's rounding.
#include <type_traits>

#include "encoder.h"
#include "encoder_common.h"

namespace kfac {
namespace {

constexpr uint32_t kOOB = 0x80000000u;   // buffer offset past every range: loads return 0

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------- activation --

// q = 1 / (1 + exp(-x)) and p = 1 - q, each to its own relative precision, of any x.
struct Logistic {
    float q, p;
    __device__ __forceinline__ explicit Logistic(float x) {
        const float e = expf(-fabsf(x)), r = 1.0f / (1.0f + e);
        q = x >= 0.0f ? r : e * r;
        p = x >= 0.0f ? e * r : r;
    }
};

// act(g) and, where asked for, its derivative.
template <bool SLOPE>
__device__ __forceinline__ float act(int kind, float g, float& slope) {
    switch (kind) {
        case kActRelu:
            if (SLOPE) slope = g > 0.0f ? 1.0f : 0.0f;
            return g < 0.0f ? 0.0f : g;
        case kActSilu: {
            const Logistic l(g);
            if (SLOPE) slope = l.q * (1.0f + g * l.p);
            return g * l.q;
        }
        case kActSigmoid: {
            const Logistic l(g);
            if (SLOPE) slope = l.q * l.p;
            return l.q;
        }
        case kActGelu: {
            const float q = 0.5f * erfcf(-0.70710678118654752f * g);
            if (SLOPE) slope = q + g * 0.39894228040143268f * expf(-0.5f * g * g);
            return g * q;
        }
        default: {   // 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))
            const Logistic l(1.5957691216057308f * g * (1.0f + 0.044715f * g * g));
            const float t = l.q * l.p;
            // (far out, where t is 0, g^2 may be infinite)
            if (SLOPE) slope = l.q + (t == 0.0f ? 0.0f : g * t * 1.5957691216057308f * (1.0f + 0.134145f * g * g));
            return g * l.q;
        }
    }
}

// ---------------------------------------------------------------- operands --

// A slab of R rows (of the output's index) by BK reduction steps in LDS, one
// plane.  KC: rows of BK elements; else BK rows of R elements.  The 16-byte
// chunks of an LDS row are permuted by the row's number so that the lanes
// read at the same time fall on different banks (16 rows at one chunk, or 4
// rows at 4 neighbouring chunks).
template <int R, int BK, bool KC>
struct Slab {
    static constexpr int PITCH = 2 * (KC ? BK : R), CH = PITCH / 16, BYTES = 2 * R * BK;
    static_assert(KC ? CH == 8 || CH == 4 : CH >= 16, "a permutation for each form");
    static __device__ __forceinline__ int swz(int row) {
        if constexpr (CH == 4) return (row >> 2) & 3;
        else if constexpr (CH == 8) return (((row >> 1) & 1) << 2) | (((row >> 2) & 1) << 1) | ((row >> 3) & 1);
        else return ((row & 3) << 2) | ((row >> 2) & 3);
    }
    static __device__ __forceinline__ int at(int row, int chunk) { return row * PITCH + ((chunk ^ swz(row)) << 4); }

    // This lane's place in a fragment: output index first + lane % 32, steps 8 (lane / 32) .. + 7.
    // The block of 32 at `first` and the step group are exclusive-or'ed on.
    struct Lane {
        int lo;
        __device__ __forceinline__ explicit Lane(int lane) {
            if constexpr (KC) {
                lo = at(lane & 31, lane >> 5);
            } else {
                const int g = lane >> 4, p = lane & 15;
                lo = at(8 * (g >> 1) + (p >> 2), 2 * (g & 1) + ((p & 3) >> 1)) + (p & 1) * 8;
            }
        }
    };
    // block: the index / 32; s: steps 16 s ..
    static __device__ __forceinline__ bf16x8 frag(const char* lds, const Lane& l, int block, int s) {
        if constexpr (KC) {
            return *reinterpret_cast<const bf16x8*>(lds + block * 32 * PITCH + (l.lo ^ (s << 5)));
        } else {
            const char* p = lds + s * 16 * PITCH;
            const int lo = l.lo ^ (block << 6);
            auto rd = [&](int a) {
                return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) short4v*)const_cast<char*>(p + a));
            };
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(rd(lo), rd((lo ^ 16) + 4 * PITCH), 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

// The first `n` (0 .. 8) elements of a fragment, zeros behind.
__device__ __forceinline__ bf16x8 first_of(bf16x8 f, int n) {
    uint4v q = __builtin_bit_cast(uint4v, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = 2 * e + 1 < n ? q[e] : 2 * e < n ? q[e] & 0xffffu : 0u;
    return __builtin_bit_cast(bf16x8, q);
}

// Copies of an operand's slabs by all THREADS threads.
template <int R, int BK, bool KC, int PL, int THREADS, bool PAIR>
struct Feed {
    using S = Slab<R, BK, KC>;
    static constexpr int COPIES = S::BYTES / 16 / THREADS;
    static_assert(COPIES * 16 * THREADS == S::BYTES, "whole copies");
    static constexpr int PIECES = COPIES * PL;
    uint32_t off[COPIES];
    int chunk;               // KC: this thread's chunk of a row (the same in every copy)
    const char* base;        // where the next slab begins
    int64_t plane;
    int64_t range;           // bytes from base to the end of the operand
    int step, wave;

    // Rows (KC) or columns [first, limit) of the operand; PAIR: the upper half
    // of the rows are those `apart` further.  k0: first step.
    __device__ __forceinline__ Feed(const ProdOperand& o, int first, int64_t k0, int tid)
        : plane(o.plane * 2), wave(__builtin_amdgcn_readfirstlane(tid >> 6)) {
        const int64_t lead = KC ? (int64_t)first * o.ld + k0 : k0 * o.ld + first;
        base = reinterpret_cast<const char*>(o.p) + lead * 2;
        range = o.bytes - lead * 2;
        step = KC ? BK * 2 : BK * o.ld * 2;
        chunk = 0;
#pragma unroll
        for (int c = 0; c < COPIES; ++c) {
            const int q = c * THREADS + tid, row = q / S::CH, ch = (q % S::CH) ^ S::swz(row);
            if constexpr (KC) {
                constexpr int H = R / 2;
                const int in = PAIR ? row % H : row;
                off[c] = first + in < o.limit ? (uint32_t)((in + (PAIR && row >= H ? o.apart : 0)) * o.ld + ch * 8) * 2 : kOOB;
                chunk = ch;
                static_assert((THREADS / S::CH) % 16 == 0, "one chunk for all copies of a thread");
            } else {
                off[c] = first + ch * 8 < o.limit ? (uint32_t)(row * o.ld + ch * 8) * 2 : kOOB;
            }
        }
    }
    // Copy `piece` of the next slab, of which `left` steps exist.
    __device__ __forceinline__ void copy(char* lds, int piece, int left) const {
        const int pl = piece / COPIES, c = piece % COPIES;
        const char* p = base + pl * plane;
        int64_t n = range;
        uint32_t o = off[c];
        if constexpr (KC) {
            if (left < BK) o |= chunk * 8 < left ? 0u : kOOB;
        } else {
            // (no steps past the end: the rows there read as zero)
            n = min(n, (int64_t)max(min(left, BK), 0) * (step / BK));
        }
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(p), (short)0, (int)max((int64_t)0, min(n, (int64_t)0x7ffffffc)), 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void*)(lds + pl * S::BYTES + (c * THREADS + wave * 64) * 16), 16, o, 0, 0, 0);
    }
    __device__ __forceinline__ void next() {
        base += step;
        range -= step;
    }
};

// ----------------------------------------------------------------- product --

constexpr int kForward = 0, kPlain = 1;   // epilogues

template <int TM_, int TN_, int WM_, int WN_, int BK_, int PL_, bool KCA_, bool KCB_, int EPI_>
struct Form {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, BK = BK_, PL = PL_, EPI = EPI_;
    static constexpr bool KCA = KCA_, KCB = KCB_;
    static constexpr int THREADS = 64 * WM * WN, MB = TM / WM / 32, NB = TN / WN / 32;
    using SA = Slab<TM, BK, KCA>;
    using SB = Slab<TN, BK, KCB>;
    static constexpr int BYTES_A = SA::BYTES * PL, BYTES_B = SB::BYTES * PL;
};
constexpr int threads_of(int wm, int wn) { return 64 * wm * wn; }

template <typename O>
__device__ __forceinline__ void put(void* out, int64_t at, float v) {
    *as_global(static_cast<O*>(out) + at) = (O)v;
}

template <class F>
__device__ __forceinline__ void product(const ProdArgs& P, char* (&As)[2], char* (&Bs)[2]) {
    constexpr int MB = F::MB, NB = F::NB, BK = F::BK, PL = F::PL;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave / F::WN, wn = wave % F::WN;
    const int64_t item = xcd_remap(blockIdx.x, gridDim.x);
    const int split = (int)(item / P.tiles), t = (int)(item % P.tiles);
    // bands of eight tile rows, column by column
    const int band = t / (8 * P.tiles_n), in = t % (8 * P.tiles_n);
    const int high = min(8, P.tiles_m - 8 * band);
    const int m0 = (8 * band + in % high) * F::TM, n0 = in / high * (F::EPI == kForward ? F::TN / 2 : F::TN);
    const int64_t k_begin = (int64_t)split * P.kchunk, k_end = min(P.K, k_begin + P.kchunk);

    floatx16 acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;

    using FA = Feed<F::TM, BK, F::KCA, PL, F::THREADS, false>;
    using FB = Feed<F::TN, BK, F::KCB, PL, F::THREADS, F::EPI == kForward>;
    FA fa(P.a, m0, k_begin, threadIdx.x);
    FB fb(P.b, n0, k_begin, threadIdx.x);
    const typename F::SA::Lane la(lane);
    const typename F::SB::Lane lb(lane);
    // a wave's blocks: forward, gate columns and the same up columns
    auto block_b = [&](int b) {
        if constexpr (F::EPI == kForward) return (b < NB / 2 ? 0 : F::TN / 64) + wn * (NB / 2) + b % (NB / 2);
        else return wn * NB + b;
    };
    auto copy_all = [&](int buf, int left) {
#pragma unroll
        for (int p = 0; p < FA::PIECES; ++p) fa.copy(As[buf], p, left);
#pragma unroll
        for (int p = 0; p < FB::PIECES; ++p) fb.copy(Bs[buf], p, left);
        fa.next();
        fb.next();
    };
    auto multiply = [&](int buf, int left, auto tail) {
#pragma unroll
        for (int s = 0; s < BK / 16; ++s) {
            bf16x8 a[PL][MB], b[PL][NB];
            const int n = left - 16 * s - 8 * (lane >> 5);   // this lane's steps
#pragma unroll
            for (int p = 0; p < PL; ++p) {
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    a[p][i] = F::SA::frag(As[buf] + p * F::SA::BYTES, la, wm * MB + i, s);
                    if (decltype(tail)::value && F::KCA) a[p][i] = first_of(a[p][i], n);
                }
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    b[p][j] = F::SB::frag(Bs[buf] + p * F::SB::BYTES, lb, block_b(j), s);
                    if (decltype(tail)::value && F::KCB) b[p][j] = first_of(b[p][j], n);
                }
            }
            // the products of parts, the smallest first
#pragma unroll
            for (int sum = PL - 1; sum >= 0; --sum)
#pragma unroll
                for (int p = 0; p <= sum; ++p)
#pragma unroll
                    for (int i = 0; i < MB; ++i)
#pragma unroll
                        for (int j = 0; j < NB; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[sum - p][i], b[p][j], acc[i][j], 0, 0, 0);
        }
    };
    int left = (int)(k_end - k_begin);
    auto turn = [&](int buf) {
        // the copies of this buffer are the only ones in flight
        __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
        __syncthreads();
        if (left > BK) copy_all(buf ^ 1, left - BK);
        if (left >= BK) multiply(buf, left, std::false_type());
        else multiply(buf, left, std::true_type());
        left -= BK;
    };
    if (left > 0) copy_all(0, left);
    while (left > 0) {
        turn(0);
        if (left <= 0) break;
        turn(1);
    }

    // lane: column lane % 32 of a block, rows 8 (r / 4) + 4 (lane / 32) + r % 4
    const int row0 = m0 + wm * MB * 32 + 4 * (lane >> 5), col = lane & 31;
    if constexpr (F::EPI == kForward) {
#pragma unroll
        for (int j = 0; j < NB / 2; ++j) {
            const int c = n0 + 32 * block_b(j) + col;
            if (c >= P.width) continue;
            const float bg = P.bias ? *as_global(P.bias + c) : 0.0f, bu = P.bias ? *as_global(P.bias + P.width + c) : 0.0f;
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t m = row0 + 32 * i + 8 * (r >> 2) + (r & 3);
                    if (m >= P.M) continue;
                    const float g = acc[i][j][r] + bg, u = acc[i][j + NB / 2][r] + bu;
                    float slope;
                    const float h = act<false>(P.act, g, slope) * u;
                    if (P.out_bf16) {
                        put<__bf16>(P.out, m * P.width + c, h);
                        if (P.pre) {
                            put<__bf16>(P.pre, m * 2 * P.width + c, g);
                            put<__bf16>(P.pre, m * 2 * P.width + P.width + c, u);
                        }
                    } else {
                        put<float>(P.out, m * P.width + c, h);
                        if (P.pre) {
                            put<float>(P.pre, m * 2 * P.width + c, g);
                            put<float>(P.pre, m * 2 * P.width + P.width + c, u);
                        }
                    }
                }
        }
    } else {
        float* part = P.part ? P.part + (int64_t)split * P.M * P.N : nullptr;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int c = n0 + 32 * block_b(j) + col;
            if (c >= P.N) continue;
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t m = row0 + 32 * i + 8 * (r >> 2) + (r & 3);
                    if (m >= P.M) continue;
                    if (part) *as_global(part + m * P.N + c) = acc[i][j][r];
                    else if (P.out_bf16) put<__bf16>(P.out, m * P.N + c, acc[i][j][r]);
                    else put<float>(P.out, m * P.N + c, acc[i][j][r]);
                }
        }
    }
}

template <int TM, int TN, int WM, int WN, int BK, int PL, bool KCA, bool KCB, int EPI>
__global__ __launch_bounds__(threads_of(WM, WN)) void product_kernel(ProdArgs P) {
    using F = Form<TM, TN, WM, WN, BK, PL, KCA, KCB, EPI>;
    __shared__ __attribute__((aligned(16))) char A0[F::BYTES_A];
    __shared__ __attribute__((aligned(16))) char A1[F::BYTES_A];
    __shared__ __attribute__((aligned(16))) char B0[F::BYTES_B];
    __shared__ __attribute__((aligned(16))) char B1[F::BYTES_B];
    char* As[2] = {A0, A1};
    char* Bs[2] = {B0, B1};
    product<F>(P, As, Bs);
}

// Adds the shares of a split product in order.
template <typename O>
__global__ __launch_bounds__(256) void product_sum_kernel(const float* part, int splits, int64_t n, void* out) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= n) return;
    const int count = (int)min((int64_t)4, n - at);
    float v[4];
    if (count == 4) {
        Vec<float>::open(v, *(const __attribute__((address_space(1))) loose16*)(part + at));
#pragma unroll 4
        for (int k = 1; k < splits; ++k) {
            float w[4];
            Vec<float>::open(w, *(const __attribute__((address_space(1))) loose16*)(part + k * n + at));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += w[e];
        }
    } else {
        for (int e = 0; e < count; ++e) {
            v[e] = *as_global(part + at + e);
            for (int k = 1; k < splits; ++k) v[e] += *as_global(part + k * n + at + e);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < count) put<O>(out, at + e, v[e]);
}

// ------------------------------------------------------------- preparation --

// Operands as the products read them: bfloat16 rows from odd widths to a
// pitch of 16 bytes, float32 rows as three planes of bfloat16 parts, columns
// past the width zero.  A part is the rest rounded to nearest, at most
// bfloat16's largest number (x0 + x1 + x2 = x down to 2^-126 or so; a part
// below that may come out of the product as zero).
__global__ __launch_bounds__(256) void repack_kernel(RepackTable T) {
    int k = 0;
    for (int i = 1; i < T.n; ++i)
        if (T.m[i].begin <= blockIdx.x) k = i;
    const RepackMatrix& R = T.m[k];
    const int64_t u = (blockIdx.x - R.begin) * 256 + threadIdx.x, groups = R.pitch / 8;
    if (u >= R.rows * groups) return;
    const int64_t row = u / groups;
    const int c = (int)(u % groups) * 8;
    __bf16* out = static_cast<__bf16*>(R.dst) + row * R.pitch + c;
    float v[8];
    auto read = [&](auto kind) {
        constexpr bool SHORT = decltype(kind)::value;
        if (R.bf16) {
            RowVec<__bf16, SHORT> q;
            q.get(static_cast<const __bf16*>(R.src) + row * R.cols, c, R.cols);
            q.open(v);
        } else {
            RowVec<float, SHORT> q[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) q[h].get(static_cast<const float*>(R.src) + row * R.cols, c + 4 * h, R.cols);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[4];
                q[h].open(w);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * h + e] = w[e];
            }
        }
    };
    if (R.cols >= 8) read(std::false_type());
    else read(std::true_type());
    if (R.bf16) {
        store_some<__bf16>(out, v, 8);
        return;
    }
    float part[3][8];
    const float most = __uint_as_float(0x7f7f0000u), all = __uint_as_float(0x7f7fffffu);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float x = v[e];
        const bool finite = fabsf(x) <= all;   // what is not goes into the first part alone
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            const float r = (float)(__bf16)x;
            part[q][e] = finite ? __builtin_amdgcn_fmed3f(r, -most, most) : q == 0 ? x : 0.0f;
            x -= part[q][e];
        }
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) store_some<__bf16>(out + q * R.plane, part[q], 8);
}

// ------------------------------------------------------ activation backward --

// dpre = [dh u act'(g) | dh act(g)] and, per workgroup, the sums of its rows
// (before dpre is rounded).  A lane keeps its columns, the four waves take
// rows in turn.
template <typename T, bool SHORT>
__global__ __launch_bounds__(256) void gated_grad_kernel(GatedGradArgs A) {
    constexpr int N = Vec<T>::N;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = (blockIdx.x * 64 + lane) * N, left = A.width - c;
    const int64_t begin = (int64_t)blockIdx.y * A.chunk, end = min(A.rows, begin + A.chunk);
    float sg[N], su[N];
#pragma unroll
    for (int e = 0; e < N; ++e) sg[e] = su[e] = 0.0f;
    if (left > 0) {
        const T* dh = static_cast<const T*>(A.dh);
        const T* pre = static_cast<const T*>(A.pre);
        T* dpre = static_cast<T*>(A.dpre) + c;
        // the next row is on its way while this one is formed
        RowVec<T, SHORT> rd, rg, ru;
        auto fetch = [&](int64_t row) {
            rd.get(dh + row * A.width, c, A.width);
            rg.get(pre + row * 2 * A.width, c, A.width);
            ru.get(pre + row * 2 * A.width + A.width, c, A.width);
        };
        if (begin + wave < end) fetch(begin + wave);
        for (int64_t row = begin + wave; row < end; row += 4) {
            float d[N], g[N], u[N];
            rd.open(d);
            rg.open(g);
            ru.open(u);
            if (row + 4 < end) fetch(row + 4);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float slope;
                const float a = act<true>(A.act, g[e], slope);
                g[e] = d[e] * u[e] * slope;
                u[e] = d[e] * a;
                sg[e] += g[e];
                su[e] += u[e];
            }
            store_some<T>(dpre + row * 2 * A.width, g, left);
            store_some<T>(dpre + row * 2 * A.width + A.width, u, left);
        }
    }
    if (A.part == nullptr) return;
    __shared__ float sums[2][N][256];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        sums[0][e][threadIdx.x] = sg[e];
        sums[1][e][threadIdx.x] = su[e];
    }
    __syncthreads();
    float* part = A.part + (int64_t)blockIdx.y * 2 * A.pitch;
    for (int k = wave; k < 2 * N; k += 4) {
        const int which = k / N, e = k % N;
        const float* s = sums[which][e] + lane;
        if (e < left) *as_global(part + which * A.pitch + c + e) = ((s[0] + s[64]) + s[128]) + s[192];
    }
}

template <int EPI, bool KCA, bool KCB>
hipError_t launch_form(const ProdArgs& a, int64_t items, bool parts, hipStream_t stream) {
    const dim3 grid((unsigned)items);
    // forward, a wave holds gate columns and their up columns: 32 of each
    constexpr int WM = EPI == kForward ? 4 : 2;
    if (parts) hipLaunchKernelGGL((product_kernel<128, 128, WM, 8 / WM, 32, 3, KCA, KCB, EPI>), grid, dim3(512), 0, stream, a);
    else hipLaunchKernelGGL((product_kernel<128, 128, 2, 2, 64, 1, KCA, KCB, EPI>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product(const ProdArgs& a, int kind, bool parts, int64_t items, hipStream_t stream) {
    if (kind == kProdForward) return launch_form<kForward, true, true>(a, items, parts, stream);
    if (kind == kProdInput) return launch_form<kPlain, true, false>(a, items, parts, stream);
    return launch_form<kPlain, false, false>(a, items, parts, stream);
}

hipError_t launch_product_sum(const float* part, int splits, int64_t n, void* out, bool bf16, hipStream_t stream) {
    const dim3 grid((unsigned)((n + 1023) / 1024));
    if (bf16) hipLaunchKernelGGL(product_sum_kernel<__bf16>, grid, dim3(256), 0, stream, part, splits, n, out);
    else hipLaunchKernelGGL(product_sum_kernel<float>, grid, dim3(256), 0, stream, part, splits, n, out);
    return hipGetLastError();
}

hipError_t launch_repack(const RepackTable& t, int64_t blocks, hipStream_t stream) {
    hipLaunchKernelGGL(repack_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, t);
    return hipGetLastError();
}

hipError_t launch_gated_grad(const GatedGradArgs& a, int parts, bool bf16, hipStream_t stream) {
    const int per = 64 * (bf16 ? 8 : 4);
    const dim3 grid((unsigned)((a.width + per - 1) / per), (unsigned)parts);
    const bool few = a.width < 8;   // rows shorter than a vector
    if (bf16 && few) hipLaunchKernelGGL((gated_grad_kernel<__bf16, true>), grid, dim3(256), 0, stream, a);
    else if (bf16) hipLaunchKernelGGL((gated_grad_kernel<__bf16, false>), grid, dim3(256), 0, stream, a);
    else if (few) hipLaunchKernelGGL((gated_grad_kernel<float, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((gated_grad_kernel<float, false>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace kfac
