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
// BK reduction steps are copied from memory straight into a ring of LDS
// buffers while the oldest is multiplied.  Half of a forward tile's columns
// are gate columns and half the same up columns, each wave holding some of
// both, so that act(g) u is formed where the sums are.  Tiles of a last round
// that would not fill the card are shared out along the reduction and their
// shares added in order by a launch of its own (no atomics).
//
// float32 operands are split into three bfloat16 parts beforehand (the
// parts add up to the number exactly) and enter as six products, which carry
// a float32 product's rounding; float32 dpre against bfloat16 x and W as three.
//
// Measured (medians of a kernel trace, operands from memory), bfloat16: forward
// 25088 x 2304 -> 4608 1057 us (1008 TFLOP/s; bound by LDS reads and products
// alike), 4096 x 1024 -> 2730 67 (2.7 rounds of tiles, 0.7 of each tile's time in
// products); dx and dW of these 1768 us (1206 TFLOP/s) and 119.  float32, 4096 x
// 1024 -> 2730: 268 forward, 476 backward (six products: 1026 and 1155 TFLOP/s of
// them); float32 dpre against bfloat16, three products: 274, and of 25088 x 2304
// -> 4608 6506 (983).
#include <type_traits>

#include "encoder.h"
#include "encoder_common.h"

namespace kfac {
namespace {

constexpr uint32_t kOOB = 0x80000000u;   // buffer offset past every range: loads return 0

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------- activation --

// The exponential of -|x| as a power of two.  The product with log2(e) is
// rounded, which by itself costs as many bits as it is large (up to 1e-5 of a
// tail): what the rounding left out, and the factor's own, goes into a
// first-order term.  FULL: with that term.  A bfloat16 output is formed without
// it (1e-5 is a four-hundredth of its half step; with it the forward pass of
// 4096 x 1024 -> 2730 took 68.1 us by gelu_tanh and 65.2 by gelu, without 62.1
// and 64.2); the backward pass, whose bias gradient is float32 and which waits
// for memory, always with it.
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;
constexpr float kFarLogistic = 256.0f, kFarNormal = 16.0f;   // past which the exponential is 0 (infinities have no remainder)

__device__ __forceinline__ float at_most(float x, float most) { return x > most ? most : x; }   // (NaN stays)

// q = 1 / (1 + exp(-x)) and p = 1 - q, each to its own relative precision, of
// any x (and of x + low): FULL, within 7 half steps of float32, 4.2e-7, from 1 down to
// the least normal number (exp2 and the reciprocal are off by a step each).
template <bool FULL>
struct Logistic {
    float q, p;
    __device__ __forceinline__ explicit Logistic(float x) {
        const float a = at_most(fabsf(x), kFarLogistic), t = -kLog2e * a;
        init(x, t, FULL ? fmaf(-kLog2eLow, a, fmaf(-kLog2e, a, -t)) : 0.0f);
    }
    __device__ __forceinline__ Logistic(float x, float low) {
        const float a = at_most(fabsf(x), kFarLogistic), t = -kLog2e * a;
        init(x, t, FULL ? fmaf(-kLog2e, x >= 0.0f ? low : -low, fmaf(-kLog2eLow, a, fmaf(-kLog2e, a, -t))) : 0.0f);
    }
    __device__ __forceinline__ void init(float x, float t, float rest) {
        float e = __builtin_exp2f(t);
        if constexpr (FULL) e = fmaf(e, kLn2 * rest, e);
        const float r = __builtin_amdgcn_rcpf(1.0f + e);
        q = x >= 0.0f ? r : e * r;
        p = x >= 0.0f ? e * r : r;
    }
};

// Phi(g) of the normal distribution, and its density times sqrt(2 pi).  The
// tail Phi(-|g|) is e = exp(-g^2 / 2) times a smooth function of |g|, here a
// polynomial in t = 1 / (1 + 0.45 |g|), fitted for the least relative error
// over |g| <= 14.5 (past which e is 0 in float32) by reweighted least squares
// at Chebyshev points: 3.5e-8, and 3e-7 evaluated in float32.  FULL, e
// carries the remainders of g^2 and of its product: the tail is within 12 half
// steps, 7e-7, down to the least normal number.
template <bool FULL>
struct Normal {
    float q, e;
    __device__ __forceinline__ explicit Normal(float g) {
        const float a = at_most(fabsf(g), kFarNormal), s = a * a, m = -0.5f * kLog2e * s;
        e = __builtin_amdgcn_exp2f(m);
        if constexpr (FULL) {
            const float rest = fmaf(-0.5f * kLog2e, fmaf(a, a, -s), fmaf(-0.5f * kLog2eLow, s, fmaf(-0.5f * kLog2e, s, -m)));
            e = fmaf(e, kLn2 * rest, e);
        }
        const float t = __builtin_amdgcn_rcpf(fmaf(0.45f, a, 1.0f));
        float r = 0.0382795185f;
        r = fmaf(r, t, -0.225619689f);
        r = fmaf(r, t, 0.5375157f);
        r = fmaf(r, t, -0.61148262f);
        r = fmaf(r, t, 0.263683498f);
        r = fmaf(r, t, -0.0216226112f);
        r = fmaf(r, t, 0.162542611f);
        r = fmaf(r, t, 0.177000687f);
        r = fmaf(r, t, 0.17970866f);
        r = fmaf(r, t, -5.77849505e-06f);
        r *= e;
        q = g >= 0.0f ? 1.0f - r : r;
    }
};

// z = 2 sqrt(2 / pi) (g + 0.044715 g^3) of |g| <= kFarNormal (others: that of
// the border, whose logistic function is 0 or 1 in float32), and what its
// roundings left out: a logistic function of z takes |z| times z's error.
struct TanhArgument {
    float z, low;
    __device__ __forceinline__ explicit TanhArgument(float g) {
        constexpr float A = 1.59576917f, AL = -4.53406805e-8f, B = 0.0713548139f, BL = 2.39883247e-9f;
        const float c = g >= 0.0f ? at_most(g, kFarNormal) : -at_most(-g, kFarNormal);
        const float s = c * c, sl = fmaf(c, c, -s), p = B * s, pl = fmaf(B, s, -p);
        const float most = p > A ? p : A, least = p > A ? A : p;
        const float w = most + least;
        const float wl = ((most - w) + least) + (pl + fmaf(B, sl, fmaf(BL, s, AL)));
        z = c * w;
        low = fmaf(c, wl, fmaf(c, w, -z));
    }
};

// act(g) and, where asked for, its derivative.
template <int KIND, bool SLOPE, bool FULL>
__device__ __forceinline__ float act(float g, float& slope) {
    if constexpr (KIND == kActRelu) {
        if (SLOPE) slope = g > 0.0f ? 1.0f : 0.0f;
        return g < 0.0f ? 0.0f : g;
    } else if constexpr (KIND == kActSilu) {
        const Logistic<FULL> l(g);
        if (SLOPE) slope = l.q * (1.0f + g * l.p);
        return g * l.q;
    } else if constexpr (KIND == kActSigmoid) {
        const Logistic<FULL> l(g);
        if (SLOPE) slope = l.q * l.p;
        return l.q;
    } else if constexpr (KIND == kActGelu) {
        const Normal<FULL> n(g);
        if (SLOPE) slope = fmaf(g * 0.39894228f, n.e, n.q);
        return g * n.q;
    } else {   // 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))
        const TanhArgument z(g);
        const Logistic<FULL> l(z.z, z.low);
        const float t = l.q * l.p;
        // (far out, where t is 0, g^2 may be infinite)
        if (SLOPE) slope = l.q + (t == 0.0f ? 0.0f : g * t * 1.5957691216057308f * (1.0f + 0.134145f * g * g));
        return g * l.q;
    }
}

// f(the activation's number as a constant)
template <typename F>
__device__ __forceinline__ void with_act(int kind, F f) {
    switch (kind) {
        case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
        case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
        case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); break;
        case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
        default: f(std::integral_constant<int, kActSigmoid>());
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
    // lo: the lane's place, from lds on; block: the index / 32 (from the
    // wave's first, which for columns is a multiple of the wave's blocks);
    // s: steps 16 s ..
    static __device__ __forceinline__ bf16x8 frag(const char* lds, int place, int block, int s) {
        if constexpr (KC) {
            return *reinterpret_cast<const bf16x8*>(lds + block * 32 * PITCH + (place ^ (s << 5)));
        } else {
            const char* p = lds + s * 16 * PITCH;
            const int lo = place ^ (block << 6);
            auto rd = [&](int a) {
                return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) short4v*)const_cast<char*>(p + a));
            };
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(rd(lo), rd((lo ^ 16) + 4 * PITCH), 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)reinterpret_cast<uintptr_t>(p); }

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
    int range;               // KC: bytes from base to the end of what the tile reads; else the bytes of a row
    int lead, step, wave;    // lead: bytes in front of the tile's columns

    // Rows (KC) or columns [first, limit) of the operand; PAIR: the upper half
    // of the rows are those `apart` further.  k0: first step.
    __device__ __forceinline__ Feed(const ProdOperand& o, int first, int64_t k0, int tid)
        : plane(o.plane * 2), wave(__builtin_amdgcn_readfirstlane(tid >> 6)) {
        const int64_t at = KC ? (int64_t)first * o.ld + k0 : k0 * o.ld + first;
        base = reinterpret_cast<const char*>(o.p) + at * 2;
        step = KC ? BK * 2 : BK * o.ld * 2;
        lead = first * 2;
        chunk = 0;
        if (KC) {
            // a tile's rows lie within 2^31 bytes
            const int64_t rest = o.bytes - at * 2, most = (int64_t)(R + (PAIR ? o.apart : 0)) * o.ld * 2;
            range = __builtin_amdgcn_readfirstlane((int)min(rest, most));
        } else {
            range = o.ld * 2;
        }
#pragma unroll
        for (int c = 0; c < COPIES; ++c) {
            const int q = c * THREADS + tid, row = q / S::CH, ch = (q % S::CH) ^ S::swz(row);
            if constexpr (KC) {
                constexpr int H = R / 2;
                const int in = PAIR ? row % H : row;
                off[c] = in < o.limit - first ? (uint32_t)((in + (PAIR && row >= H ? o.apart : 0)) * o.ld + ch * 8) * 2 : kOOB;
                chunk = ch;
                static_assert((THREADS / S::CH) % 16 == 0, "one chunk for all copies of a thread");
            } else {
                off[c] = ch * 8 < o.limit - first ? (uint32_t)(row * o.ld + ch * 8) * 2 : kOOB;
            }
        }
    }
    // All copies of the next slab, of which `left` steps exist; the others read
    // as zero.  Written out: the compiler, which cannot tell the buffers
    // apart across the loop, would let the LDS reads of one wait for the
    // copies to the other.  For the same reason it does not name the memory that
    // it writes: the barriers do, and none of the buffer's reads can cross them.
    __device__ __forceinline__ void copy(char* lds, int left) {
        const int n = KC ? max(range, 0) : max(min(left, BK) * range - lead, 0);
#pragma unroll
        for (int pl = 0; pl < PL; ++pl) {
            const uint64_t p = (uint64_t)(base + pl * plane);
            const uint4v rs = {(uint32_t)p, (uint32_t)(p >> 32) & 0xffffu, (uint32_t)n, 0x00020000u};
#pragma unroll
            for (int c = 0; c < COPIES; ++c) {
                const uint32_t o = KC ? off[c] | (chunk * 8 < left ? 0u : kOOB) : off[c];
                const uint32_t to = lds_addr(lds + pl * S::BYTES + (c * THREADS + wave * 64) * 16);
                asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                             :
                             : "s"(to), "v"(o), "s"(rs)
                             : "m0");
            }
        }
        base += step;
        if (KC) range -= step;
    }
    // Rows of the reduction index: a slab whose steps end inside a 16-byte
    // chunk holds another row's elements there; they become zero.
    static __device__ __forceinline__ void clear_end(char* lds, int left, int tid) {
        if constexpr (KC) {
#pragma unroll
            for (int n = 0; n < R * PL; n += THREADS) {
                const int row = (n + tid) % R, pl = (n + tid) / R;
                if (n + tid >= R * PL) break;
                uint16_t* p = reinterpret_cast<uint16_t*>(lds + pl * S::BYTES + S::at(row, left / 8));
                for (int e = left % 8; e < 8; ++e) p[e] = 0;
            }
        }
    }
};

// ----------------------------------------------------------------- product --

constexpr int kForward = 0, kPlain = 1;   // epilogues

// PA, PB: bfloat16 parts of an operand's elements, 1 or 3.  Of three parts each,
// the six products that reach float32's rounding; of three and one, all three.
template <int TM_, int TN_, int WM_, int WN_, int BK_, int RING_, int PA_, int PB_, bool KCA_, bool KCB_, int EPI_>
struct Form {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, BK = BK_, RING = RING_, PA = PA_, PB = PB_, EPI = EPI_;
    static constexpr int PARTS = PA > PB ? PA : PB, PAIRS = PA == 3 && PB == 3 ? 6 : PARTS;
    static constexpr bool KCA = KCA_, KCB = KCB_;
    static constexpr int THREADS = 64 * WM * WN, MB = TM / WM / 32, NB = TN / WN / 32;
    // matrix-core steps of 16 whose operands are read at once
    static constexpr int SUB = PARTS == 1 && MB * NB <= 4 && BK == 64 ? 2 : 1;
    using SA = Slab<TM, BK, KCA>;
    using SB = Slab<TN, BK, KCB>;
    static constexpr int BYTES_A = SA::BYTES * PA, BYTES_B = SB::BYTES * PB;
};
constexpr int threads_of(int wm, int wn) { return 64 * wm * wn; }

// vmcnt(n) alone (expcnt and lgkmcnt left at their maximum)
__device__ __forceinline__ constexpr int vmcnt_imm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// Order of a step for the scheduler: its products, each with a share of the
// next operands' LDS reads in its shadow.
template <class F>
__device__ __forceinline__ void interleave() {
    constexpr int PRODUCTS = F::SUB * F::MB * F::NB * F::PAIRS;
    constexpr int READS = F::SUB * (F::PA * F::MB * (F::KCA ? 1 : 2) + F::PB * F::NB * (F::KCB ? 1 : 2));
    constexpr int EACH = (READS + PRODUCTS - 1) / PRODUCTS;
#pragma unroll
    for (int n = 0; n < PRODUCTS; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, EACH, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Row and column of a tile: bands of eight tile rows, column by column, so
// that the tiles of neighbouring items share operands.
__device__ __forceinline__ void tile_place(const ProdArgs& P, int t, int& row, int& col) {
    const int band = t / (8 * P.tiles_n), in = t % (8 * P.tiles_n);
    const int high = min(8, P.tiles_m - 8 * band);
    row = 8 * band + in % high;
    col = in / high;
}

// Tile t of a product, or share `split` of its reduction.
template <class F>
__device__ __forceinline__ void product(const ProdArgs& P, char* lds, int t, int split, bool shared) {
    constexpr int MB = F::MB, NB = F::NB, BK = F::BK, PA = F::PA, PB = F::PB;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave / F::WN, wn = wave % F::WN;
    int m0, n0;
    tile_place(P, t, m0, n0);
    m0 *= F::TM;   // (with what lies past it in the tile, up to 2^31 + 254: a row of its own is 64 bits wide)
    n0 *= F::EPI == kForward ? F::TN / 2 : F::TN;
    const int64_t k_begin = (int64_t)split * P.kchunk, k_end = shared ? min(P.K, k_begin + P.kchunk) : P.K;

    floatx16 acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.0f;

    using FA = Feed<F::TM, BK, F::KCA, PA, F::THREADS, false>;
    using FB = Feed<F::TN, BK, F::KCB, PB, F::THREADS, F::EPI == kForward>;
    FA fa(P.a, m0, k_begin, threadIdx.x);
    FB fb(P.b, n0, k_begin, threadIdx.x);
    constexpr int HALF = F::TN / 64;   // forward: from a block of gate columns to the same up columns
    // this lane's places in the slabs of a buffer
    int pa = typename F::SA::Lane(lane).lo, pb = F::BYTES_A + typename F::SB::Lane(lane).lo;
    if constexpr (F::KCA) pa += wm * MB * 32 * F::SA::PITCH;
    else pa ^= (wm * MB) << 6;
    constexpr int OWN = F::EPI == kForward ? NB / 2 : NB;
    if constexpr (F::KCB) pb += wn * OWN * 32 * F::SB::PITCH;
    else pb ^= (wn * OWN) << 6;
    // RING buffers, one multiplied and the others on their way; two sets of
    // operands, one in the products and one on its way from LDS.
    constexpr int SUB = F::SUB, STEPS = BK / (16 * SUB), BUFFER = F::BYTES_A + F::BYTES_B, RING = F::RING, COPIES = FA::PIECES + FB::PIECES;
    static_assert((RING - 1) * COPIES < 64, "the copies in flight can be counted");
    static_assert(STEPS % 2 == 0, "a slab begins with the first set");
    bf16x8 oa[2][SUB][PA][MB], ob[2][SUB][PB][NB];
    auto read = [&](int set, int at, int step) {
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            const int s = step * SUB + u;
#pragma unroll
            for (int p = 0; p < F::PARTS; ++p) {
#pragma unroll
                for (int i = 0; p < PA && i < MB; ++i) oa[set][u][p][i] = F::SA::frag(lds + p * F::SA::BYTES, pa + at, i, s);
#pragma unroll
                for (int j = 0; p < PB && j < NB; ++j)
                    ob[set][u][p][j] = F::SB::frag(lds + p * F::SB::BYTES, pb + at, j < OWN ? j : HALF + j - OWN, s);
            }
        }
    };
    auto multiply = [&](int set) {
        // the products of parts, the smallest first
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int sum = F::PARTS - 1; sum >= 0; --sum)
#pragma unroll
                for (int p = 0; p <= sum && p < PB; ++p)
#pragma unroll
                    for (int i = 0; sum - p < PA && i < MB; ++i)
#pragma unroll
                        for (int j = 0; j < NB; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(oa[set][u][sum - p][i], ob[set][u][p][j],
                                                                                acc[i][j], 0, 0, 0);
    };
    // added to the sums at the end; on its way from here on
    float bias[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) bias[b] = 0.0f;
    if constexpr (F::EPI == kForward) {
        if (P.bias != nullptr && !shared) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int col = min(n0 + (wn * OWN + b % OWN) * 32 + (lane & 31), P.width - 1);
                bias[b] = *as_global(P.bias + (b < OWN ? 0 : P.width) + col);
            }
        }
    }
    int left = __builtin_amdgcn_readfirstlane((int)(k_end - k_begin));
    auto copy = [&](int at, int n) {
        fa.copy(lds + at, n);
        fb.copy(lds + at + F::BYTES_A, n);
    };
    auto clear = [&](int at, int n) {
        if ((F::KCA || F::KCB) && n > 0 && n < BK && n % 8 != 0) {
            FA::clear_end(lds + at, n, threadIdx.x);
            FB::clear_end(lds + at + F::BYTES_A, n, threadIdx.x);
            lds_barrier();
        }
    };
    if (left > 0) {
        // (a descriptor's words may have come from the vector unit, which a load must not follow at once)
        asm volatile("s_nop 4");
#pragma unroll
        for (int n = 0; n < RING; ++n) copy(n * BUFFER, left - n * BK);
        __builtin_amdgcn_s_waitcnt(vmcnt_imm((RING - 1) * COPIES));
        asm volatile("s_barrier" ::: "memory");
        clear(0, left);
        read(0, 0, 0);
        // One slab a turn.  Its last operands are in registers before its last
        // products: the barrier stands there, behind the copies of the next
        // slab, so that the next slab's first operands are read beside those
        // products, and another slab is copied over this one.  (Copies past
        // the end read nothing, and are not branched around.)
        int at = 0;
        do {
            const int next = at + BUFFER < RING * BUFFER ? at + BUFFER : 0;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (s + 1 < STEPS) {
                    read((s + 1) & 1, at, s + 1);
                } else {
                    __builtin_amdgcn_s_waitcnt(vmcnt_imm((RING - 2) * COPIES) & 0xf0ff);   // and lgkmcnt(0)
                    asm volatile("s_barrier" ::: "memory");
                    clear(next, left - BK);
                    read(0, next, 0);
                    copy(at, left - RING * BK);
                }
                multiply(s & 1);
                interleave<F>();
            }
            at = next;
            left -= BK;
        } while (left > 0);
        // the copies past the end, which read nothing, still write zeros
        __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
    }

    // The sums go through LDS, 32 rows of the wave's columns at a time (lane:
    // column lane % 32 of a block, rows 8 (r / 4) + 4 (lane / 32) + r % 4), so
    // that a lane holds eight neighbouring columns of a row and writes them at
    // once; two rows at a time, for the reads of one beside the other's work.
    constexpr int PITCH = NB * 32 + 4, CHUNKS = OWN * 4, TURNS = CHUNKS / 2;
    static_assert(F::WM * F::WN * 32 * PITCH * 4 <= RING * BUFFER, "a stretch of LDS for each wave");
    static_assert(TURNS % 2 == 0, "two rows at a time");
    asm volatile("s_barrier" ::: "memory");
    float* stage = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
    // this lane's columns, the same in every turn
    const int c8 = lane % CHUNKS * 8, col = n0 + wn * OWN * 32 + c8, have = (F::EPI == kForward ? P.width : P.N) - col;
    const bool inside = F::TM <= P.M - m0 && n0 + (F::EPI == kForward ? F::TN / 2 : F::TN) <= (F::EPI == kForward ? P.width : P.N);
    using O = typename std::conditional<PB == 1, __bf16, float>::type;   // (the type of x and of the weights)
    auto write = [&](auto* out, const float (&v)[8], bool there) {
        using T = typename std::remove_pointer<decltype(out)>::type;
        constexpr int N = Vec<T>::N;
#pragma unroll
        for (int k = 0; k < 8; k += N) {
            float q[N];
#pragma unroll
            for (int e = 0; e < N; ++e) q[e] = v[k + e];
            if (inside) store_all<T>(out + k, q);
            else if (there) store_some<T>(out + k, q, have - k);
        }
    };
#pragma unroll
    for (int i = 0; i < MB; ++i) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                stage[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * PITCH + 32 * j + (lane & 31)] = acc[i][j][r] + bias[j];
#pragma unroll 1
        for (int q = 0; q < TURNS; q += 2) {
            float v[2][8], w[2][8];
            int64_t m[2];
            bool there[2];
            int row[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                row[h] = ((q + h) * 64 + lane) / CHUNKS;
                m[h] = (int64_t)m0 + (wm * MB + i) * 32 + row[h];
                there[h] = m[h] < P.M && have > 0;
                const float* from = stage + row[h] * PITCH + c8;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[h][e] = from[e];
                if constexpr (F::EPI == kForward) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[h][e] = from[OWN * 32 + e];
                }
            }
            if (shared) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float* part = P.part + ((int64_t)split * (P.tiles - P.whole) + (t - P.whole)) * (F::TM * F::TN) +
                                  ((wm * MB + i) * 32 + row[h]) * F::TN + wn * OWN * 32 + c8;
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        store_all<float>(part + e, {v[h][e], v[h][e + 1], v[h][e + 2], v[h][e + 3]});
                        if constexpr (F::EPI == kForward)
                            store_all<float>(part + F::TN / 2 + e, {w[h][e], w[h][e + 1], w[h][e + 2], w[h][e + 3]});
                    }
                }
            } else if constexpr (F::EPI == kForward) {
                if (P.pre) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        O* pre = static_cast<O*>(P.pre) + m[h] * 2 * P.width + col;
                        write(pre, v[h], there[h]);
                        write(pre + P.width, w[h], there[h]);
                    }
                }
                with_act(P.act, [&](auto kind) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float slope;
                            v[h][e] = act<decltype(kind)::value, false, PB != 1>(v[h][e], slope) * w[h][e];
                        }
                });
#pragma unroll
                for (int h = 0; h < 2; ++h) write(static_cast<O*>(P.out) + m[h] * P.width + col, v[h], there[h]);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (PB == 1 && P.out_bf16) write(static_cast<__bf16*>(P.out) + m[h] * P.N + col, v[h], there[h]);
                    else write(static_cast<float*>(P.out) + m[h] * P.N + col, v[h], there[h]);
                }
            }
        }
    }
}

template <int TM, int TN, int WM, int WN, int BK, int RING, int PL>
__global__ __launch_bounds__(threads_of(WM, WN)) void gated_forward_kernel(ProdArgs P) {
    using F = Form<TM, TN, WM, WN, BK, RING, PL, PL, true, true, kForward>;
    __shared__ __attribute__((aligned(16))) char lds[RING * (F::BYTES_A + F::BYTES_B)];
    // whole tiles, then shares
    const bool shared = (int)blockIdx.x >= P.whole;
    const int rest = P.tiles - P.whole;
    const int b = shared ? (int)xcd_remap(blockIdx.x - P.whole, gridDim.x - P.whole) : (int)xcd_remap(blockIdx.x, P.whole);
    product<F>(P, lds, shared ? P.whole + b % rest : b, shared ? b / rest : 0, shared);
}

// The tiles that were shared out: their shares in order, then the bias and the
// activation; four neighbouring columns of both projections a thread.
template <int TM, int TN, typename T>
__global__ __launch_bounds__(256) void gated_forward_finish_kernel(ProdArgs A) {
    constexpr int LANES = TN / 8, ROWS = 256 / LANES, EACH = TM / ROWS, TILE = TM * TN;
    const int rest = A.tiles - A.whole, u = blockIdx.x / EACH;
    const int i = blockIdx.x % EACH * ROWS + threadIdx.x / LANES, j = threadIdx.x % LANES * 4;
    int tm, tn;
    tile_place(A, A.whole + u, tm, tn);
    const int64_t m = (int64_t)tm * TM + i;
    const int n = tn * (TN / 2) + j;
    const int have = A.width - n;
    if (m >= A.M || have <= 0) return;
    const float* p = A.part + (int64_t)u * TILE + i * TN + j;
    float v[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) Vec<float>::open(v[h], *as_global(reinterpret_cast<const uint4v*>(p + h * (TN / 2))));
#pragma unroll 4
    for (int s = 1; s < A.splits; ++s) {
        float w[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            Vec<float>::open(w[h], *as_global(reinterpret_cast<const uint4v*>(p + (int64_t)s * rest * TILE + h * (TN / 2))));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h][e] += w[h][e];
    }
    T* pre = A.pre ? static_cast<T*>(A.pre) + m * 2 * A.width + n : nullptr;
    T* out = static_cast<T*>(A.out) + m * A.width + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (e >= have) break;
        float g = v[0][e], q = v[1][e];
        if (A.bias) {
            g += *as_global(A.bias + n + e);
            q += *as_global(A.bias + A.width + n + e);
        }
        if (pre) {
            *as_global(pre + e) = (T)g;
            *as_global(pre + A.width + e) = (T)q;
        }
        with_act(A.act, [&](auto kind) {
            float slope;
            g = act<decltype(kind)::value, false, std::is_same<T, float>::value>(g, slope) * q;
        });
        *as_global(out + e) = (T)g;
    }
}

// The forward product of few rows: what counts then is how fast the weights
// come.  A workgroup holds 16 gate columns and the same up columns of 16 MB
// rows; its eight waves share the reduction and read their stretches of the
// weights' rows straight into the operands of 16 x 16 blocks, and their sums
// meet in LDS.  float32 operands enter as they are (v_mfma_f32_16x16x4: rates
// do not count here), a lane's four steps one by one: both operands agree on
// the order, which is all that a sum needs.
template <typename T, int MB, bool SHORT>
__global__ __launch_bounds__(64 * kRowsWaves) void gated_rows_kernel(RowsArgs A) {
    constexpr int WAVES = kRowsWaves, N = Vec<T>::N, UNIT = 4 * N, DEEP = 4;   // steps of one block product, and those read at once
    typedef float floatx4 __attribute__((ext_vector_type(4)));
    __shared__ float sums[WAVES][2 * MB * 4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16, i = lane & 15, k = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 16 * MB;
    // this lane's rows; those past the end repeat the last one
    const int n = min(n0 + i, A.width - 1);
    const T* gate = static_cast<const T*>(A.weight) + (int64_t)n * A.d;
    const T* up = gate + (int64_t)A.width * A.d;
    const T* x[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) x[b] = static_cast<const T*>(A.x) + min(m0 + 16 * b + i, A.rows - 1) * A.d;
    const int units = (A.d + UNIT - 1) / UNIT, each = (units + WAVES - 1) / WAVES;
    const int first = wave * each, last = min(units, first + each);
    floatx4 acc[2][MB];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[p][b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int u = first; u < last; u += DEEP) {
        RowVec<T, SHORT> w[DEEP][2], v[DEEP][MB];
        const bool ends = (u + DEEP) * UNIT > A.d;
#pragma unroll
        for (int e = 0; e < DEEP; ++e) {
            // (a turn past the wave's last unit reads the row's end, which is cut to nothing)
            const int at = u + e < last ? (u + e) * UNIT + k * N : units * UNIT + k * N;
            w[e][0].get(gate, at, A.d);
            w[e][1].get(up, at, A.d);
#pragma unroll
            for (int b = 0; b < MB; ++b) v[e][b].get(x[b], at, A.d);
        }
        const bool cut = ends || u + DEEP > last;
#pragma unroll
        for (int e = 0; e < DEEP; ++e) {
            const uint4v g = w[e][0].raw(cut), p = w[e][1].raw(cut);
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                const uint4v r = v[e][b].raw(cut);
                if constexpr (N == 8) {
                    const bf16x8 xr = __builtin_bit_cast(bf16x8, r);
                    acc[0][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xr, __builtin_bit_cast(bf16x8, g), acc[0][b], 0, 0, 0);
                    acc[1][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xr, __builtin_bit_cast(bf16x8, p), acc[1][b], 0, 0, 0);
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        acc[0][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(r[t]), __uint_as_float(g[t]), acc[0][b], 0, 0, 0);
                        acc[1][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(r[t]), __uint_as_float(p[t]), acc[1][b], 0, 0, 0);
                    }
                }
            }
        }
    }
    // lane: column lane % 16, rows 4 (lane / 16) + r
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) sums[wave][(p * MB + b) * 4 + r][lane] = acc[p][b][r];
    __syncthreads();
    for (int e = wave; e < MB * 4; e += WAVES) {
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int s = 0; s < WAVES; ++s) {
            g += sums[s][e][lane];
            u += sums[s][MB * 4 + e][lane];
        }
        const int64_t m = m0 + 16 * (e >> 2) + 4 * k + (e & 3);
        const int c = n0 + i;
        if (m >= A.rows || c >= A.width) continue;
        if (A.bias) {
            g += *as_global(A.bias + c);
            u += *as_global(A.bias + A.width + c);
        }
        if (A.pre) {
            T* pre = static_cast<T*>(A.pre) + m * 2 * A.width + c;
            *as_global(pre) = (T)g;
            *as_global(pre + A.width) = (T)u;
        }
        with_act(A.act, [&](auto kind) {
            float slope;
            g = act<decltype(kind)::value, false, std::is_same<T, float>::value>(g, slope) * u;
        });
        *as_global(static_cast<T*>(A.h) + m * A.width + c) = (T)g;
    }
}

// dx and dW in one launch, so that the one's last round is the other's first:
// whole tiles of dx, of dW, then the shares of each.  (The longest first
// would be better by some percent where dW's reduction is the longer one.)
// Slabs of 64 or 32 steps, two or three, for each of the two, 4096 rows of
// 1024 -> 2 x 2730, operands from memory / from the caches: 64 and 64 110 / 107 us,
// 32 and 32 120 / 106, 64 and 32 114 / 104; 2048 rows 66, 64 and 63 (dx reads
// rows of dpre in pieces of a slab's length, dW 256 bytes either way).  By
// 256 x 256, 25088 rows of 2304 -> 2 x 4608: 64 and 64 1809, 64 and 32 1760, 32
// and 32 1731 to 1760.
template <int TM, int TN, int WM, int WN, int BKX, int RINGX, int BKW, int RINGW, int PA, int PB>
__global__ __launch_bounds__(threads_of(WM, WN)) void gated_backward_kernel(ProdPair P) {
    using FX = Form<TM, TN, WM, WN, BKX, RINGX, PA, PB, true, false, kPlain>;
    using FW = Form<TM, TN, WM, WN, BKW, RINGW, PA, PB, false, false, kPlain>;
    constexpr int BYTES_X = RINGX * (FX::BYTES_A + FX::BYTES_B), BYTES_W = RINGW * (FW::BYTES_A + FW::BYTES_B);
    __shared__ __attribute__((aligned(16))) char lds[BYTES_X > BYTES_W ? BYTES_X : BYTES_W];
    int b = (int)blockIdx.x, which = 0;
    // ranges of items: whole tiles of both, shares of both
    bool shared = false;
    int count = P.p[0].whole;
#pragma unroll
    for (int k = 1; k < 4; ++k) {
        if (b < count) break;
        b -= count;
        which = k & 1;
        shared = k >= 2;
        count = shared ? (P.p[which].tiles - P.p[which].whole) * P.p[which].splits : P.p[which].whole;
    }
    b = (int)xcd_remap(b, count);
    auto run = [&](auto form, const ProdArgs& A) {
        const int rest = A.tiles - A.whole;
        product<decltype(form)>(A, lds, shared ? A.whole + b % rest : b, shared ? b / rest : 0, shared);
    };
    if (which == 0) run(FX(), P.p[0]);
    else run(FW(), P.p[1]);
}

// What the backward pass leaves to add up, 256 threads a workgroup: the tiles
// that were shared out, their shares in order (four neighbouring elements a
// thread), and the bias's gradient.  88 tiles of 128 x 128 in five shares: 8.5 us.
template <int TM, int TN>
__global__ __launch_bounds__(256) void gated_finish_kernel(ProdPair P, PartSums S) {
    constexpr int ROWS = 1024 / TN, EACH = TM / ROWS, TILE = TM * TN;
    int b = (int)blockIdx.x;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const ProdArgs& A = P.p[k];
        const int rest = A.splits > 1 ? A.tiles - A.whole : 0;
        if (b >= rest * EACH) {
            b -= rest * EACH;
            continue;
        }
        const int u = b / EACH, i = b % EACH * ROWS + threadIdx.x / (TN / 4), j = threadIdx.x % (TN / 4) * 4;
        int tm, tn;
        tile_place(A, A.whole + u, tm, tn);
        const int64_t m = (int64_t)tm * TM + i;
        const int n = tn * TN + j;
        if (m >= A.M || n >= A.N) return;
        const float* p = A.part + (int64_t)u * TILE + i * TN + j;
        float v[4];
        Vec<float>::open(v, *as_global(reinterpret_cast<const uint4v*>(p)));
#pragma unroll 4
        for (int s = 1; s < A.splits; ++s) {
            float w[4];
            Vec<float>::open(w, *as_global(reinterpret_cast<const uint4v*>(p + (int64_t)s * rest * TILE)));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += w[e];
        }
        const int64_t at = m * A.N + n;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e >= A.N) break;
            if (A.out_bf16) *as_global(static_cast<__bf16*>(A.out) + at + e) = (__bf16)v[e];
            else *as_global(static_cast<float*>(A.out) + at + e) = v[e];
        }
        return;
    }
    __shared__ float join[4][kSumColumns];
    add_parts<float>(S, b, join);
}

// ------------------------------------------------------------- preparation --

// Three bfloat16 parts of float32 numbers, each the rest rounded to nearest, at
// most bfloat16's largest number.
template <int N>
__device__ __forceinline__ void split_parts(const float (&v)[N], float (&part)[3][N]) {
    const float most = __uint_as_float(0x7f7f0000u), all = __uint_as_float(0x7f7fffffu);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        float x = v[e];
        const bool finite = fabsf(x) <= all;   // what is not goes into the first part alone
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            const float r = (float)(__bf16)x;
            part[q][e] = finite ? __builtin_amdgcn_fmed3f(r, -most, most) : q == 0 ? x : 0.0f;
            x -= part[q][e];
        }
    }
}

// Operands as the products read them: bfloat16 rows from odd widths to a
// pitch of 16 bytes, float32 rows as three planes of bfloat16 parts, columns
// past the width zero.  (x0 + x1 + x2 = x down to 2^-126 or so; a part below
// that may come out of the product as zero.)  9.8 million float32 elements: 21 us,
// 4.7 TB/s.
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
    split_parts(v, part);
#pragma unroll
    for (int q = 0; q < 3; ++q) store_some<__bf16>(out + q * R.plane, part[q], 8);
}

// ------------------------------------------------------ activation backward --

// N numbers as D, of which `count` have a place.
template <typename D, int N>
__device__ __forceinline__ void store_row(D* p, const float (&v)[N], int count) {
    constexpr int M = Vec<D>::N;
#pragma unroll
    for (int k = 0; k < N; k += M) {
        float q[M];
#pragma unroll
        for (int e = 0; e < M; ++e) q[e] = v[k + e];
        store_some<D>(p + k, q, count - k);
    }
}

// Up to four numbers as bfloat16, at any element.
__device__ __forceinline__ void store_bf16x4(uint16_t* p, const float (&v)[4], int count) {
    typedef uint32_t loose8 __attribute__((ext_vector_type(2), aligned(2)));
    const uint32_t lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(floatx2{v[0], v[1]}, bf16x2));
    const uint32_t hi = __builtin_bit_cast(uint32_t, __builtin_convertvector(floatx2{v[2], v[3]}, bf16x2));
    if (count >= 4) {
        *(__attribute__((address_space(1))) loose8*)p = loose8{lo, hi};
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < count) *as_global(p + e) = (uint16_t)((e < 2 ? lo : hi) >> (16 * (e & 1)));
    }
}

// dpre = [dh u act'(g) | dh act(g)] and, per workgroup, the sums of its rows
// (before dpre is rounded).  A lane keeps its columns, the four waves take
// rows in turn.  Bound by memory: 25088 x 4608 bfloat16 224 us (5.2 TB/s), 4096 x
// 2730 27 (4.1 TB/s, rows that begin on any 4 bytes); with float32 dpre and its
// three planes 685 and 84.
template <typename T, typename D, bool SHORT>
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
        D* dpre = static_cast<D*>(A.dpre) + c;
        // whether this workgroup's columns reach past the row's end
        const bool ends = ((int)blockIdx.x + 1) * 64 * N > A.width;
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
            rd.open(d, ends);
            rg.open(g, ends);
            ru.open(u, ends);
            if (row + 4 < end) fetch(row + 4);
            with_act(A.act, [&](auto kind) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    float slope;
                    const float a = act<decltype(kind)::value, true, true>(g[e], slope);
                    g[e] = d[e] * u[e] * slope;
                    u[e] = d[e] * a;
                    sg[e] += g[e];
                    su[e] += u[e];
                }
            });
            store_row<D>(dpre + row * 2 * A.width, g, left);
            store_row<D>(dpre + row * 2 * A.width + A.width, u, left);
            if constexpr (std::is_same<D, float>::value) {
                // the products' operand as well
                if (A.planes == nullptr) continue;
                uint16_t* to = A.planes + row * A.plane_pitch + c;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float part[3][N];
                    split_parts(h ? u : g, part);
#pragma unroll
                    for (int q = 0; q < 3; ++q)
#pragma unroll
                        for (int k = 0; k < N; k += 4)
                            store_bf16x4(to + q * A.plane + h * A.width + k, {part[q][k], part[q][k + 1], part[q][k + 2], part[q][k + 3]},
                                         left - k);
                }
            }
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

}  // namespace

hipError_t launch_gated_forward(const ProdArgs& a, int form, int64_t items, hipStream_t stream) {
    const dim3 grid((unsigned)items);
    switch (form) {
        case kProdWide: hipLaunchKernelGGL((gated_forward_kernel<256, 256, 2, 4, 64, 2, 1>), grid, dim3(512), 0, stream, a); break;
        case kProdPair: hipLaunchKernelGGL((gated_forward_kernel<128, 128, 2, 2, 64, 2, 1>), grid, dim3(256), 0, stream, a); break;
        case kProdDeep: hipLaunchKernelGGL((gated_forward_kernel<128, 128, 2, 2, 64, 3, 1>), grid, dim3(256), 0, stream, a); break;
        // a wave holds gate columns and their up columns, 32 of each
        default: hipLaunchKernelGGL((gated_forward_kernel<128, 128, 4, 2, 32, 3, 3>), grid, dim3(512), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_gated_forward_finish(const ProdArgs& a, int form, hipStream_t stream) {
    const int m = kProdForms[form].m, n = kProdForms[form].n;
    const dim3 grid((unsigned)((int64_t)(a.tiles - a.whole) * (m * n / 2048)));
    if (form == kProdWide) hipLaunchKernelGGL((gated_forward_finish_kernel<256, 256, __bf16>), grid, dim3(256), 0, stream, a);
    else if (form != kProdParts) hipLaunchKernelGGL((gated_forward_finish_kernel<128, 128, __bf16>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((gated_forward_finish_kernel<128, 128, float>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <typename T, bool SHORT>
hipError_t launch_rows(const RowsArgs& a, hipStream_t stream) {
    const int blocks = gated_rows_blocks(a.rows);
    const dim3 grid((unsigned)((a.width + 15) / 16), (unsigned)((a.rows + 16 * blocks - 1) / (16 * blocks)));
    if (blocks == 1) hipLaunchKernelGGL((gated_rows_kernel<T, 1, SHORT>), grid, dim3(64 * kRowsWaves), 0, stream, a);
    else if (blocks == 2) hipLaunchKernelGGL((gated_rows_kernel<T, 2, SHORT>), grid, dim3(64 * kRowsWaves), 0, stream, a);
    else hipLaunchKernelGGL((gated_rows_kernel<T, 4, SHORT>), grid, dim3(64 * kRowsWaves), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_gated_rows(const RowsArgs& a, bool bf16, hipStream_t stream) {
    const bool few = a.d < 8;   // rows shorter than a vector
    if (bf16) return few ? launch_rows<__bf16, true>(a, stream) : launch_rows<__bf16, false>(a, stream);
    return few ? launch_rows<float, true>(a, stream) : launch_rows<float, false>(a, stream);
}

hipError_t launch_gated_backward(const ProdPair& a, int form, int64_t items, hipStream_t stream) {
    const dim3 grid((unsigned)items);
    switch (form) {
        case kProdWide: hipLaunchKernelGGL((gated_backward_kernel<256, 256, 2, 4, 32, 4, 32, 4, 1, 1>), grid, dim3(512), 0, stream, a); break;
        case kProdPair: hipLaunchKernelGGL((gated_backward_kernel<128, 128, 2, 2, 64, 2, 32, 3, 1, 1>), grid, dim3(256), 0, stream, a); break;
        case kProdDeep: hipLaunchKernelGGL((gated_backward_kernel<128, 128, 2, 2, 64, 3, 64, 3, 1, 1>), grid, dim3(256), 0, stream, a); break;
        case kProdMixed: hipLaunchKernelGGL((gated_backward_kernel<128, 128, 2, 2, 32, 2, 32, 2, 3, 1>), grid, dim3(256), 0, stream, a); break;
        default: hipLaunchKernelGGL((gated_backward_kernel<128, 128, 2, 4, 32, 3, 32, 3, 3, 3>), grid, dim3(512), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_gated_finish(const ProdPair& a, int form, const PartSums& s, hipStream_t stream) {
    const int m = kProdForms[form].m, n = kProdForms[form].n, each = m * n / 1024;
    int64_t blocks = s.dweight || s.dbias ? sums_blocks(s.pitch) : 0;
    for (const ProdArgs& p : a.p) blocks += p.splits > 1 ? (int64_t)(p.tiles - p.whole) * each : 0;
    if (blocks == 0) return hipSuccess;
    const dim3 grid((unsigned)blocks);
    if (n == 256) hipLaunchKernelGGL((gated_finish_kernel<256, 256>), grid, dim3(256), 0, stream, a, s);
    else hipLaunchKernelGGL((gated_finish_kernel<128, 128>), grid, dim3(256), 0, stream, a, s);
    return hipGetLastError();
}

hipError_t launch_repack(const RepackTable& t, int64_t blocks, hipStream_t stream) {
    hipLaunchKernelGGL(repack_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, t);
    return hipGetLastError();
}

template <typename T, typename D>
hipError_t launch_grad(const GatedGradArgs& a, int parts, hipStream_t stream) {
    const int per = 64 * Vec<T>::N;
    const dim3 grid((unsigned)((a.width + per - 1) / per), (unsigned)parts);
    // (rows shorter than a vector)
    if (a.width < 8) hipLaunchKernelGGL((gated_grad_kernel<T, D, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((gated_grad_kernel<T, D, false>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_gated_grad(const GatedGradArgs& a, int parts, bool bf16, bool dpre_bf16, hipStream_t stream) {
    if (!bf16) return launch_grad<float, float>(a, parts, stream);
    return dpre_bf16 ? launch_grad<__bf16, __bf16>(a, parts, stream) : launch_grad<__bf16, float>(a, parts, stream);
}

}  // namespace kfac
