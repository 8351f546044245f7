// Attention of an encoder layer, forward and backward, with a learned
// relative position bias by buckets.
//
//   s_ij = scale q_i . k_j + bias[bucket(j - p_i)],  p_i = i + len_k - len_q
//   forward   P = softmax_j(s), out_i = sum_j P_ij v_j, lse_i = log sum_j exp s_ij
//   backward  P_ij = exp(s_ij - lse_i) again, dP = dout v^T, delta_i = dout_i . out_i,
//             dS = P (dP - delta), dq = scale dS k, dk = scale dS^T q, dv = P^T dout,
//             dbias[n] = sum of dS over the pairs of bucket n
//
// All products run on 32 x 32 matrix-core blocks.  The scores are formed as
// S^T (rows = keys) where a wave owns queries, and as S (rows = queries)
// where it owns keys: the wave's own index is then the block's column, which
// is fixed per lane, and the sixteen rows of a lane's column are the
// reduction index of the next product.  A reduction may be taken in any
// order, so the block's registers serve as the next product's operand as
// they are, and the other operand is read in the same order (rows 4 g .. + 3
// and 8 + 4 g .. + 3 of each 16 for lane half g).  The probabilities never
// leave the registers, and the softmax statistics of a query take one
// exchange between the two halves of the wave.
//
// The backward pass runs twice over the scores, once by keys (dK, dV) and
// once by queries (dQ and the bias gradient), so that every sum has one
// owner and one order: no atomics, the same bits on every run.
#include <type_traits>

#include "device_common.h"
#include "training.h"

namespace kfac {
namespace {

constexpr int NT = kAttnThreads;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kOOB = 0x80000000u;   // buffer offset past every range: loads return 0

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));

// A fragment holds 8 values of the reduction index per lane: for bf16 one
// matrix-core operand, for float32 eight of v_mfma_f32_32x32x2_f32 (value t
// of both lane halves is instruction t's pair; the two operands agree on the
// order, which is all that a sum needs).
template <typename T>
struct Ops;
template <>
struct Ops<__bf16> {
    using Frag = bf16x8;
    static __device__ __forceinline__ void mma(floatx16& c, const Frag& a, const Frag& b) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // registers 8 s .. 8 s + 7 of a block, rounded to nearest even
    static __device__ __forceinline__ Frag from(const floatx16& x, int s) {
        union {
            Frag f;
            bf16x2 h[4];
        } u;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const floatx2 v = {x[8 * s + 2 * t], x[8 * s + 2 * t + 1]};
            u.h[t] = __builtin_convertvector(v, bf16x2);
        }
        return u.f;
    }
};
template <>
struct Ops<float> {
    using Frag = floatx8;
    static __device__ __forceinline__ void mma(floatx16& c, const Frag& a, const Frag& b) {
#pragma unroll
        for (int t = 0; t < 8; ++t) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[t], b[t], c, 0, 0, 0);
    }
    static __device__ __forceinline__ Frag from(const floatx16& x, int s) {
        Frag f;
#pragma unroll
        for (int t = 0; t < 8; ++t) f[t] = x[8 * s + t];
        return f;
    }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, 0x7fffffff, 0x00020000);
}

// A tile of ROWS rows in LDS, DC columns of T in rows of DS (a power of
// two).  The 16-byte chunks of a row are permuted by the row's number so
// that 16 consecutive rows read at one chunk, and 4 consecutive rows read at
// 4 neighbouring chunks (the transposing reads), fall on different banks:
// with 4 or 2 rows per 256 bytes of banks the rows' own position already
// separates them, and the low bits of what is left go to the chunk's high
// bits.
template <typename T, int DC, int ROWS>
struct Tile {
    static constexpr int ES = sizeof(T);
    static constexpr int DS = DC <= 32 ? 32 : DC <= 64 ? 64 : 128;
    static constexpr int PITCH = DS * ES;         // bytes per row
    static constexpr int CH = PITCH / 16;         // chunks per row
    static constexpr int CHC = DC * ES / 16;      // chunks in use
    static constexpr int BYTES = ROWS * PITCH;
    static constexpr int COPIES = (ROWS * CHC + NT - 1) / NT;
    using Frag = typename Ops<T>::Frag;

    static __device__ __forceinline__ int swz(int row) {
        if constexpr (CH == 4) return (row >> 2) & 3;
        else if constexpr (CH == 8) return (((row >> 1) & 1) << 2) | (((row >> 2) & 1) << 1) | ((row >> 3) & 1);
        else return ((row & 3) << 2) | ((row >> 2) & 3);
    }
    static __device__ __forceinline__ int at(int row, int chunk) { return row * PITCH + ((chunk ^ swz(row)) << 4); }

    // This thread's chunks of the tile whose row 0 is `base`: rows from
    // `rows` on and columns from `dim` on are zero.
    static __device__ __forceinline__ void load(uint4v (&r)[COPIES], const char* base, int64_t stride_bytes, int rows,
                                                int dim) {
        const __amdgpu_buffer_rsrc_t rs = rows_rsrc(base);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int idx = threadIdx.x + NT * i, row = idx / CHC, chunk = idx % CHC;
            const bool ok = row < rows && row < ROWS && chunk * (16 / ES) < dim;
            const uint32_t off = ok ? (uint32_t)(row * (int)stride_bytes + chunk * 16) : kOOB;
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
        }
    }
    static __device__ __forceinline__ void store(char* lds, const uint4v (&r)[COPIES]) {
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int idx = threadIdx.x + NT * i, row = idx / CHC, chunk = idx % CHC;
            if ((ROWS * CHC) % NT == 0 || row < ROWS) *reinterpret_cast<uint4v*>(lds + at(row, chunk)) = r[i];
        }
    }
    // Rows row0 + lane % 32, columns 16 s + 8 (lane / 32) .. + 7.
    static __device__ __forceinline__ Frag row_frag(const char* lds, int row0, int s, int lane) {
        const int row = row0 + (lane & 31), g = lane >> 5;
        if constexpr (ES == 2) {
            return *reinterpret_cast<const bf16x8*>(lds + at(row, 2 * s + g));
        } else {
            const floatx4 a = *reinterpret_cast<const floatx4*>(lds + at(row, 4 * s + 2 * g));
            const floatx4 b = *reinterpret_cast<const floatx4*>(lds + at(row, 4 * s + 2 * g + 1));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // Column col0 + lane % 32, rows row0 + 4 g .. + 3 and row0 + 8 + 4 g .. + 3 (g = lane / 32).
    static __device__ __forceinline__ Frag col_frag(const char* lds, int row0, int col0, int lane) {
        if constexpr (ES == 2) {
            const int gr = lane >> 4, p = lane & 15;
            const int col = col0 + 16 * (gr & 1) + 4 * (p & 3), row = row0 + 4 * (gr >> 1) + (p >> 2);
            auto rd = [&](int r) {
                const char* a = lds + at(r, col >> 3) + (col & 7) * 2;
                return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) short4v*)const_cast<char*>(a));
            };
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(rd(row), rd(row + 8), 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int col = col0 + (lane & 31), row = row0 + 4 * (lane >> 5);
            Frag f;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int r = row + 8 * (t >> 2) + (t & 3);
                f[t] = *reinterpret_cast<const float*>(lds + at(r, col >> 2) + (col & 3) * 4);
            }
            return f;
        }
    }
};

// This lane's row of an operand that stays in registers: columns
// 16 s + 8 (lane / 32) .. + 7 of row `row` (zero from `rows` and `dim` on).
template <typename T, int DC>
__device__ __forceinline__ void own_frags(typename Ops<T>::Frag (&f)[DC / 16], const char* base, int64_t stride_bytes,
                                          int row, int rows, int dim, int lane) {
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(base);
    const int g = lane >> 5;
#pragma unroll
    for (int s = 0; s < DC / 16; ++s) {
        const int col = 16 * s + 8 * g;
        const uint32_t off = (row < rows && col < dim) ? (uint32_t)(row * (int)stride_bytes + col * (int)sizeof(T)) : kOOB;
        if constexpr (sizeof(T) == 2) {
            f[s] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
        } else {
            const floatx4 a = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
            const floatx4 b = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(rs, off + 16, 0, 0));
            f[s] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
}

// Writes column-owned sums (block b: rows = columns 32 b .. of the tensor,
// this lane's column = tensor row `p`) times `f`.
template <typename T, int DC>
__device__ __forceinline__ void store_rows(char* p, const floatx16 (&acc)[DC / 32], float f, int dim, int lane) {
    const int g = lane >> 5;
#pragma unroll
    for (int b = 0; b < DC / 32; ++b)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int col = 32 * b + 8 * t + 4 * g;
            if (col >= dim) continue;
            const floatx4 v = {acc[b][4 * t] * f, acc[b][4 * t + 1] * f, acc[b][4 * t + 2] * f, acc[b][4 * t + 3] * f};
            if constexpr (sizeof(T) == 2) {
                union {
                    bf16x2 h[2];
                    uint2v u;
                } u;
                const floatx2 lo = {v[0], v[1]}, hi = {v[2], v[3]};
                u.h[0] = __builtin_convertvector(lo, bf16x2);
                u.h[1] = __builtin_convertvector(hi, bf16x2);
                *as_global(reinterpret_cast<uint2v*>(p + col * 2)) = u.u;
            } else {
                *as_global(reinterpret_cast<floatx4*>(p + col * 4)) = v;
            }
        }
}

template <int N>
__device__ __forceinline__ void clear(floatx16 (&a)[N]) {
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) a[b][r] = 0.0f;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, 64); }

// Row of a 32 x 32 block in register r of lane half g.
__device__ __forceinline__ int block_row(int r, int g) { return 8 * (r >> 2) + 4 * g + (r & 3); }

template <typename T>
__device__ __forceinline__ char* at_row(const AttnTensor& t, int64_t b, int64_t row, int64_t h) {
    return static_cast<char*>(t.p) + (b * t.sb + row * t.sl + h * t.sh) * (int64_t)sizeof(T);
}

__device__ __forceinline__ int visible_keys(const AttnArgs& A, int b) {
    int n = A.len_k;
    if (A.lens) n = min(n, max(0, __builtin_amdgcn_readfirstlane(as_global(A.lens)[b])));
    return n;
}

// The bias of one head in log2 units.  Blocks wholly beyond the stretch of
// offsets where the bucket changes take one of two constants; the others
// look their offsets up, in LDS where the stretch is short (the workgroup
// fills the table once), else in the workspace.
struct Bias {
    const float* near;   // LDS, from offset far_lo - kAttnPad on
    const float* rel;    // workspace, at offset 0 of key - query (not position)
    float lo, hi;        // beyond far_lo and far_hi

    __device__ __forceinline__ void begin(const AttnArgs& A, float* table, int h) {
        near = table;
        rel = A.near_n ? nullptr : A.rel + h * A.rel_ld + (A.lq_pad - 1);
        lo = as_global(A.bias)[(int64_t)A.far_lo_bucket * A.heads + h] * kLog2e;
        hi = as_global(A.bias)[(int64_t)A.far_hi_bucket * A.heads + h] * kLog2e;
        for (int c = threadIdx.x; c < A.near_n; c += NT) {
            const int n = bucket_of(A.borders, A.far_lo - kAttnPad + c);
            table[c] = as_global(A.bias)[(int64_t)n * A.heads + h] * kLog2e;
        }
    }
    static __device__ __forceinline__ int bucket_of(const AttnBorders& B, int d) {
        const int dist = B.two_sided ? abs(d) : max(-d, 0);
        int n = B.two_sided && d > 0 ? B.n + 1 : 0;
        for (int k = 0; k < B.n; ++k) n += dist >= B.at[k];
        return n;
    }
    // A 32 x 32 block that is not beyond.  KEYS_ARE_ROWS: rows are keys
    // base + .., this lane's column is query `own`; else rows are queries
    // base + .., this lane's column is key `own`.  A block's offsets lie
    // within 94 of the stretch, inside the table's margin.
    template <bool KEYS_ARE_ROWS>
    __device__ __forceinline__ void block(floatx16& b, const AttnArgs& A, int base, int own, int g) const {
        const int sign = KEYS_ARE_ROWS ? 1 : -1, zero = sign * (base + 4 * g - own);
        if (A.near_n) {
            const float* p = near + (zero - (A.len_k - A.len_q) - A.far_lo + kAttnPad);
#pragma unroll
            for (int r = 0; r < 16; ++r) b[r] = p[sign * (8 * (r >> 2) + (r & 3))];
        } else {
            const float* p = rel + zero;
#pragma unroll
            for (int r = 0; r < 16; ++r) b[r] = as_global(p)[sign * (8 * (r >> 2) + (r & 3))];
        }
    }
};

// ---------------------------------------------------------------- forward --
template <typename T, int DC, bool BIAS>
__global__ __launch_bounds__(NT, 2) void attn_forward_kernel(AttnArgs A) {
    constexpr int TK = sizeof(T) == 2 ? 64 : 32;
    using Kt = Tile<T, DC, TK>;
    __shared__ __attribute__((aligned(16))) char Ks[2][Kt::BYTES];
    __shared__ __attribute__((aligned(16))) char Vs[2][Kt::BYTES];
    __shared__ float Near[BIAS ? kAttnNear : 1];
    using Frag = typename Ops<T>::Frag;
    const int64_t item = xcd_remap(blockIdx.x, gridDim.x);
    const int64_t bh = item / A.qtiles;
    const int qt = A.qtiles - 1 - (int)(item % A.qtiles);   // the longest rows of a causal head first
    const int b = (int)(bh / A.heads), h = (int)(bh % A.heads), hk = h / A.group;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), g = lane >> 5;
    const int shift = A.len_k - A.len_q;
    const int q0 = qt * kAttnRows, qw = q0 + 32 * wave, i = qw + (lane & 31);
    const int nk = visible_keys(A, b);
    // keys this workgroup, this wave and this lane's query may see
    const int last = min(A.len_q, q0 + kAttnRows) - 1;
    const int nwg = A.causal ? max(0, min(nk, last + shift + 1)) : nk;
    const int nlane = A.causal ? max(0, min(nk, i + shift + 1)) : nk;
    const int nwave_lo = A.causal ? max(0, min(nk, qw + shift + 1)) : nk;
    const int nwave_hi = qw >= A.len_q ? 0 : A.causal ? max(0, min(nk, qw + 31 + shift + 1)) : nk;

    Frag qf[DC / 16];
    own_frags<T, DC>(qf, at_row<T>(A.q, b, qw, h), A.q.sl * (int64_t)sizeof(T), lane & 31, A.len_q - qw, A.dim, lane);
    Bias table;
    if constexpr (BIAS) table.begin(A, Near, h);

    floatx16 o[DC / 32];
    clear(o);
    float m = -INFINITY, l = 0.0f;
    const int tiles = (nwg + TK - 1) / TK;
    uint4v rk[Kt::COPIES], rv[Kt::COPIES];
    auto fetch = [&](int j0) {
        Kt::load(rk, at_row<T>(A.k, b, j0, hk), A.k.sl * (int64_t)sizeof(T), nk - j0, A.dim);
        Kt::load(rv, at_row<T>(A.v, b, j0, hk), A.v.sl * (int64_t)sizeof(T), nk - j0, A.dim);
    };
    if (tiles > 0) {
        fetch(0);
        Kt::store(Ks[0], rk);
        Kt::store(Vs[0], rv);
    }
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
        const int j0 = t * TK;
        const char *K = Ks[t & 1], *V = Vs[t & 1];
        if (t + 1 < tiles) fetch(j0 + TK);
        if (j0 < nwave_hi) {
            floatx16 x[TK / 32];
            clear(x);
#pragma unroll
            for (int u = 0; u < TK / 32; ++u)
#pragma unroll
                for (int s = 0; s < DC / 16; ++s) Ops<T>::mma(x[u], Kt::row_frag(K, 32 * u, s, lane), qf[s]);
            // scores in log2 units
            const int lo = j0 - (qw + 31 + shift), hi = j0 + TK - 1 - (qw + shift);
            if (BIAS && !(lo >= A.far_hi || hi <= A.far_lo)) {
#pragma unroll
                for (int u = 0; u < TK / 32; ++u) {
                    floatx16 bias;
                    table.block<true>(bias, A, j0 + 32 * u, i, g);
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[u][r] = fmaf(x[u][r], A.scale2, bias[r]);
                }
            } else {
                const float bias = !BIAS ? 0.0f : hi <= A.far_lo ? table.lo : table.hi;
#pragma unroll
                for (int u = 0; u < TK / 32; ++u)
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[u][r] = fmaf(x[u][r], A.scale2, bias);
            }
            if (j0 + TK > nwave_lo) {
#pragma unroll
                for (int u = 0; u < TK / 32; ++u)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (j0 + 32 * u + block_row(r, g) >= nlane) x[u][r] = -INFINITY;
            }
            float top = x[0][0];
#pragma unroll
            for (int u = 0; u < TK / 32; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, x[u][r]);
            top = fmaxf(m, fmaxf(top, other_half(top)));
            const float base = top == -INFINITY ? 0.0f : top;   // a row that has seen nothing yet
            const float keep = exp2_fast(m - base);
            m = top;
            float sum = 0.0f;
#pragma unroll
            for (int u = 0; u < TK / 32; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    x[u][r] = exp2_fast(x[u][r] - base);
                    sum += x[u][r];
                }
            l = fmaf(l, keep, sum);
#pragma unroll
            for (int d = 0; d < DC / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[d][r] *= keep;
#pragma unroll
            for (int u = 0; u < TK / 32; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Frag p = Ops<T>::from(x[u], s);
#pragma unroll
                    for (int d = 0; d < DC / 32; ++d)
                        Ops<T>::mma(o[d], Kt::col_frag(V, 32 * u + 16 * s, 32 * d, lane), p);
                }
        }
        if (t + 1 < tiles) {
            Kt::store(Ks[(t + 1) & 1], rk);
            Kt::store(Vs[(t + 1) & 1], rv);
        }
        __syncthreads();
    }
    if (i >= A.len_q) return;
    l += other_half(l);
    store_rows<T, DC>(at_row<T>(A.out, b, i, h), o, l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l, A.dim, lane);
    if (g == 0) as_global(A.lse)[bh * A.len_q + i] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
}

// --------------------------------------------------------------- backward --
// dbias[n][h]: the waves' shares of head h, in the order of sequences, tiles
// and waves.  One workgroup per head and bucket; thread t sums every 256th
// share, then a tree over the threads.
__device__ __forceinline__ void sum_bias(const AttnArgs& A, float* S, int item) {
    const int h = item % A.heads, n = item / A.heads;
    const int per = A.qtiles * 4;
    const int64_t count = (int64_t)A.batch * per;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < count; c += NT) {
        const int64_t b = c / per, w = c % per;
        s += as_global(A.part)[((b * A.heads + h) * per + w) * A.buckets + n];
    }
    S[threadIdx.x] = s;
    __syncthreads();
    for (int w = NT / 2; w > 0; w /= 2) {
        if ((int)threadIdx.x < w) S[threadIdx.x] += S[threadIdx.x + w];
        __syncthreads();
    }
    if (threadIdx.x == 0) as_global(A.dbias)[(int64_t)n * A.heads + h] = S[0];
}

// dK and dV of 128 KB keys, 32 KB per wave; queries pass by in tiles of 32:
// those of one query head of the group and one chunk of its rows where the
// key tiles are shared out in parts (`parts` > 1, the shares summed by
// attn_kv_sum_kernel), else all.  The workgroups past the key tiles sum the
// bias gradient.
template <typename T, int DC, int KB, bool BIAS>
__global__ __launch_bounds__(NT, sizeof(T) == 2 && KB * DC <= 64 ? 2 : 1) void attn_dkdv_kernel(AttnArgs A) {
    constexpr int TQ = 32;
    using Qt = Tile<T, DC, TQ>;
    __shared__ __attribute__((aligned(16))) char Qs[2][Qt::BYTES];
    __shared__ __attribute__((aligned(16))) char Ds[2][Qt::BYTES];
    __shared__ __attribute__((aligned(16))) float Ls[2][2][TQ];
    __shared__ float Near[BIAS ? kAttnNear : NT];
    using Frag = typename Ops<T>::Frag;
    const int64_t tiles = (int64_t)A.batch * A.kv_heads * A.parts * A.ktiles;
    if constexpr (BIAS) {
        if (blockIdx.x >= tiles) {
            sum_bias(A, Near, (int)(blockIdx.x - tiles));
            return;
        }
    }
    // key tiles fastest: neighbours read the same queries
    const int64_t item = xcd_remap(blockIdx.x, tiles);
    const int kt = (int)(item % A.ktiles);
    const int64_t rest = item / A.ktiles;
    const int part = (int)(rest % A.parts);
    const int64_t bk = rest / A.parts;
    const int b = (int)(bk / A.kv_heads), hk = (int)(bk % A.kv_heads);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), g = lane >> 5;
    const int shift = A.len_k - A.len_q;
    const int k0 = kt * kAttnRows * KB, kw = k0 + 32 * KB * wave;
    const int nk = visible_keys(A, b);

    Frag kf[KB][DC / 16], vf[KB][DC / 16];
    floatx16 dk[KB][DC / 32], dv[KB][DC / 32];
#pragma unroll
    for (int n = 0; n < KB; ++n) {
        const int row = 32 * n + (lane & 31);
        own_frags<T, DC>(kf[n], at_row<T>(A.k, b, kw, hk), A.k.sl * (int64_t)sizeof(T), row, nk - kw, A.dim, lane);
        own_frags<T, DC>(vf[n], at_row<T>(A.v, b, kw, hk), A.v.sl * (int64_t)sizeof(T), row, nk - kw, A.dim, lane);
        clear(dk[n]);
        clear(dv[n]);
    }

    // query tiles of this part, from the first one that sees key k0 (causal: j <= i + shift)
    const int heads = A.parts > 1 ? 1 : A.group, chunks = A.parts > 1 ? A.parts / A.group : 1;
    const int h0 = hk * A.group + (A.parts > 1 ? part / chunks : 0);
    const int qtiles = (A.len_q + TQ - 1) / TQ;
    const int first = max(A.causal ? max(0, k0 - shift) / TQ : 0, part % chunks * A.qchunk);
    const int per = k0 < nk ? max(0, min(qtiles, (part % chunks + 1) * A.qchunk) - first) : 0;
    const int steps = per * heads;
    Bias table;
    uint4v rq[Qt::COPIES], rd[Qt::COPIES];
    float rl = 0.0f;
    int fh = h0, fi = first * TQ;          // head and first query of the next fetch
    auto fetch = [&]() {
        Qt::load(rq, at_row<T>(A.q, b, fi, fh), A.q.sl * (int64_t)sizeof(T), A.len_q - fi, A.dim);
        Qt::load(rd, at_row<T>(A.dout, b, fi, fh), A.dout.sl * (int64_t)sizeof(T), A.len_q - fi, A.dim);
        if (threadIdx.x < 2 * TQ) {
            const float* p = threadIdx.x < TQ ? A.lse2 : A.delta;
            rl = as_global(p)[((int64_t)b * A.heads + fh) * A.lq_pad + fi + (threadIdx.x & (TQ - 1))];
        }
        fi += TQ;
        if (fi >= (first + per) * TQ) {
            fi = first * TQ;
            ++fh;
        }
    };
    auto put = [&](int buf) {
        Qt::store(Qs[buf], rq);
        Qt::store(Ds[buf], rd);
        if (threadIdx.x < 2 * TQ) Ls[buf][threadIdx.x / TQ][threadIdx.x & (TQ - 1)] = rl;
    };
    int h = h0, i0 = first * TQ;
    if (steps > 0) {
        fetch();
        put(0);
        if constexpr (BIAS) table.begin(A, Near, h);
    }
    __syncthreads();
    for (int st = 0; st < steps; ++st) {
        const char *Q = Qs[st & 1], *D = Ds[st & 1];
        const float *L = Ls[st & 1][0], *E = Ls[st & 1][1];
        if (st + 1 < steps) fetch();
        // a wave whose keys are all hidden from these queries has nothing to add
        if (kw < nk && (!A.causal || kw <= i0 + TQ - 1 + shift)) {
            floatx16 x[KB], y[KB];
            clear(x);
            clear(y);
#pragma unroll
            for (int s = 0; s < DC / 16; ++s) {
                const Frag f = Qt::row_frag(Q, 0, s, lane);
#pragma unroll
                for (int n = 0; n < KB; ++n) Ops<T>::mma(x[n], f, kf[n][s]);
            }
#pragma unroll
            for (int s = 0; s < DC / 16; ++s) {
                const Frag f = Qt::row_frag(D, 0, s, lane);
#pragma unroll
                for (int n = 0; n < KB; ++n) Ops<T>::mma(y[n], f, vf[n][s]);
            }
#pragma unroll
            for (int n = 0; n < KB; ++n) {
                const int kn = kw + 32 * n, j = kn + (lane & 31);
                if constexpr (BIAS) {
                    const int lo = kn - (i0 + TQ - 1 + shift), hi = kn + 31 - (i0 + shift);
                    if (lo >= A.far_hi || hi <= A.far_lo) {
                        const float bias = hi <= A.far_lo ? table.lo : table.hi;
#pragma unroll
                        for (int r = 0; r < 16; ++r) x[n][r] = fmaf(x[n][r], A.scale2, bias);
                    } else {
                        floatx16 bias;
                        table.block<false>(bias, A, i0, j, g);
#pragma unroll
                        for (int r = 0; r < 16; ++r) x[n][r] = fmaf(x[n][r], A.scale2, bias[r]);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[n][r] *= A.scale2;
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const floatx4 l4 = *reinterpret_cast<const floatx4*>(L + 8 * t + 4 * g);
                    const floatx4 e4 = *reinterpret_cast<const floatx4*>(E + 8 * t + 4 * g);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        x[n][4 * t + c] = exp2_fast(x[n][4 * t + c] - l4[c]);
                        y[n][4 * t + c] = x[n][4 * t + c] * (y[n][4 * t + c] - e4[c]);
                    }
                }
                if (kn + 32 > nk || (A.causal && kn + 31 > i0 + shift)) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (j >= nk || (A.causal && j > i0 + block_row(r, g) + shift)) x[n][r] = y[n][r] = 0.0f;
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                Frag p[KB], ds[KB];
#pragma unroll
                for (int n = 0; n < KB; ++n) {
                    p[n] = Ops<T>::from(x[n], s);
                    ds[n] = Ops<T>::from(y[n], s);
                }
#pragma unroll
                for (int d = 0; d < DC / 32; ++d) {
                    const Frag fd = Qt::col_frag(D, 16 * s, 32 * d, lane), fq = Qt::col_frag(Q, 16 * s, 32 * d, lane);
#pragma unroll
                    for (int n = 0; n < KB; ++n) {
                        Ops<T>::mma(dv[n][d], fd, p[n]);
                        Ops<T>::mma(dk[n][d], fq, ds[n]);
                    }
                }
            }
        }
        if (st + 1 < steps) put((st + 1) & 1);
        i0 += TQ;
        if (i0 >= (first + per) * TQ && st + 1 < steps) {
            i0 = first * TQ;
            ++h;
            if constexpr (BIAS) {
                __syncthreads();           // every wave is done with the last head's table
                table.begin(A, Near, h);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < KB; ++n) {
        const int j = kw + 32 * n + (lane & 31);
        if (j >= A.len_k) continue;
        if (A.parts > 1) {
            const int64_t row = ((int64_t)part * A.batch * A.kv_heads + bk) * A.len_k + j;
            const int64_t all = (int64_t)A.parts * A.batch * A.kv_heads * A.len_k;
            store_rows<float, DC>(reinterpret_cast<char*>(A.kv_part + row * A.dim), dk[n], A.scale, A.dim, lane);
            store_rows<float, DC>(reinterpret_cast<char*>(A.kv_part + (all + row) * A.dim), dv[n], 1.0f, A.dim, lane);
        } else {
            store_rows<T, DC>(at_row<T>(A.dk, b, j, hk), dk[n], A.scale, A.dim, lane);
            store_rows<T, DC>(at_row<T>(A.dv, b, j, hk), dv[n], 1.0f, A.dim, lane);
        }
    }
}

// dk (blockIdx.y = 0) and dv from their shares, in the shares' order; eight
// values per thread.
template <typename T>
__global__ __launch_bounds__(NT) void attn_kv_sum_kernel(AttnArgs A) {
    const int per = A.dim / 8;
    const int64_t rows = (int64_t)A.batch * A.kv_heads * A.len_k, c = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (c >= rows * per) return;
    const int64_t row = c / per;
    const int col = (int)(c % per) * 8;
    const floatx4* p = reinterpret_cast<const floatx4*>(
        A.kv_part + ((int64_t)blockIdx.y * A.parts * rows + row) * A.dim + col);
    floatx4 lo = as_global(p)[0], hi = as_global(p)[1];
    for (int n = 1; n < A.parts; ++n) {
        p += rows * A.dim / 4;
        lo += as_global(p)[0];
        hi += as_global(p)[1];
    }
    const int64_t bk = row / A.len_k, j = row % A.len_k;
    char* o = at_row<T>(blockIdx.y ? A.dv : A.dk, bk / A.kv_heads, j, bk % A.kv_heads) + col * sizeof(T);
    if constexpr (sizeof(T) == 2) {
        typedef float floatx8_ __attribute__((ext_vector_type(8)));
        const floatx8_ v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        *as_global(reinterpret_cast<uint4v*>(o)) = __builtin_bit_cast(uint4v, __builtin_convertvector(v, bf16x8));
    } else {
        as_global(reinterpret_cast<floatx4*>(o))[0] = lo;
        as_global(reinterpret_cast<floatx4*>(o))[1] = hi;
    }
}

// The bias gradient of one 32 x 32 block of dS (rows = keys, columns =
// queries) that spans several buckets: the block goes through LDS, lane t
// sums the diagonal key - query = t - 31, and lane n adds the diagonals of
// bucket n (and n + 64) in order to its own sums.  `base` is the offset of
// the block's diagonal 0.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
constexpr int kDiagPitch = 33;
__device__ __forceinline__ void near_bias(const floatx16& ds, float* S, float* diag, int base, const int2 (&range)[2],
                                          float (&sum)[2], int lane) {
    const int g = lane >> 5;
#pragma unroll
    for (int r = 0; r < 16; ++r) S[block_row(r, g) * kDiagPitch + (lane & 31)] = ds[r];
    wave_fence();
    const int t = lane - 31;
    float d = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        const int c = r - t;
        const bool in = (unsigned)c < 32u;
        const float v = S[in ? r * kDiagPitch + c : 0];
        d += in ? v : 0.0f;
    }
    diag[lane] = d;
    wave_fence();
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int lo = max(range[n].x - base, -31), hi = min(range[n].y - base, 31);
        for (int c = lo; c <= hi; ++c) sum[n] += diag[c + 31];
    }
    wave_fence();
}

// dQ of 128 queries, 32 per wave, and the waves' shares of the bias gradient.
template <typename T, int DC, bool BIAS>
__global__ __launch_bounds__(NT, sizeof(T) == 2 ? 2 : 1) void attn_dq_kernel(AttnArgs A) {
    constexpr int TK = 32;
    using Kt = Tile<T, DC, TK>;
    __shared__ __attribute__((aligned(16))) char Ks[2][Kt::BYTES];
    __shared__ __attribute__((aligned(16))) char Vs[2][Kt::BYTES];
    __shared__ float Ss[BIAS ? 4 * 32 * kDiagPitch : 1];
    __shared__ float Dg[BIAS ? 4 * 64 : 1];
    __shared__ float Near[BIAS ? kAttnNear : 1];
    using Frag = typename Ops<T>::Frag;
    const int64_t item = xcd_remap(blockIdx.x, gridDim.x);
    const int64_t bh = item / A.qtiles;
    const int qt = A.qtiles - 1 - (int)(item % A.qtiles);
    const int b = (int)(bh / A.heads), h = (int)(bh % A.heads), hk = h / A.group;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), g = lane >> 5;
    const int shift = A.len_k - A.len_q;
    const int q0 = qt * kAttnRows, qw = q0 + 32 * wave, i = qw + (lane & 31);
    const int nk = visible_keys(A, b);
    const int last = min(A.len_q, q0 + kAttnRows) - 1;
    const int nwg = A.causal ? max(0, min(nk, last + shift + 1)) : nk;
    const int nlane = A.causal ? max(0, min(nk, i + shift + 1)) : nk;
    const int nwave_lo = A.causal ? max(0, min(nk, qw + shift + 1)) : nk;
    const int nwave_hi = qw >= A.len_q ? 0 : A.causal ? max(0, min(nk, qw + 31 + shift + 1)) : nk;

    Frag qf[DC / 16], df[DC / 16];
    own_frags<T, DC>(qf, at_row<T>(A.q, b, qw, h), A.q.sl * (int64_t)sizeof(T), lane & 31, A.len_q - qw, A.dim, lane);
    own_frags<T, DC>(df, at_row<T>(A.dout, b, qw, h), A.dout.sl * (int64_t)sizeof(T), lane & 31, A.len_q - qw, A.dim,
                     lane);
    // delta from the rows in registers, and lse in log2 units; both are kept
    // for the pass by keys.  Rows that see nothing, and rows past the last,
    // get lse = +inf, which makes every probability 0.
    float lse2 = INFINITY, delta = 0.0f;
    {
        Frag of[DC / 16];
        own_frags<T, DC>(of, at_row<T>(A.out, b, qw, h), A.out.sl * (int64_t)sizeof(T), lane & 31, A.len_q - qw, A.dim,
                         lane);
#pragma unroll
        for (int s = 0; s < DC / 16; ++s)
#pragma unroll
            for (int t = 0; t < 8; ++t) delta = fmaf((float)df[s][t], (float)of[s][t], delta);
        delta += other_half(delta);
        if (i < A.len_q) {
            const float v = as_global(A.lse)[bh * A.len_q + i];
            if (v != -INFINITY) lse2 = v * kLog2e;
        }
        if (g == 0) {
            as_global(A.lse2)[bh * A.lq_pad + i] = lse2;
            as_global(A.delta)[bh * A.lq_pad + i] = delta;
        }
    }
    Bias table;
    float near_sum[2] = {0.0f, 0.0f}, far_lo_sum = 0.0f, far_hi_sum = 0.0f;
    int2 range[2];
    if constexpr (BIAS) {
        table.begin(A, Near, h);
        // offsets (key - query position) of buckets lane and lane + 64
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            constexpr int kFar = 1 << 30;
            const int per = A.borders.n + 1, at = lane + 64 * n, side = at / per, k = at % per;
            range[n] = make_int2(kFar, -kFar);
            if (at < A.buckets) {
                const int from = k == 0 ? 0 : A.borders.at[k - 1], to = k == A.borders.n ? kFar : A.borders.at[k] - 1;
                range[n] = side ? make_int2(max(from, 1), to) : make_int2(-to, -from);
                if (!A.borders.two_sided && k == 0) range[n].y = kFar;
            }
        }
    }

    floatx16 dq[DC / 32];
    clear(dq);
    const int tiles = (nwg + TK - 1) / TK;
    uint4v rk[Kt::COPIES], rv[Kt::COPIES];
    auto fetch = [&](int j0) {
        Kt::load(rk, at_row<T>(A.k, b, j0, hk), A.k.sl * (int64_t)sizeof(T), nk - j0, A.dim);
        Kt::load(rv, at_row<T>(A.v, b, j0, hk), A.v.sl * (int64_t)sizeof(T), nk - j0, A.dim);
    };
    if (tiles > 0) {
        fetch(0);
        Kt::store(Ks[0], rk);
        Kt::store(Vs[0], rv);
    }
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
        const int j0 = t * TK;
        const char *K = Ks[t & 1], *V = Vs[t & 1];
        if (t + 1 < tiles) fetch(j0 + TK);
        if (j0 < nwave_hi) {
            floatx16 x, y;
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.0f;
#pragma unroll
            for (int s = 0; s < DC / 16; ++s) Ops<T>::mma(x, Kt::row_frag(K, 0, s, lane), qf[s]);
#pragma unroll
            for (int s = 0; s < DC / 16; ++s) Ops<T>::mma(y, Kt::row_frag(V, 0, s, lane), df[s]);
            const int lo = j0 - (qw + 31 + shift), hi = j0 + TK - 1 - (qw + shift);
            const bool near = BIAS && !(lo >= A.far_hi || hi <= A.far_lo);
            if (near) {
                floatx16 bias;
                table.block<true>(bias, A, j0, i, g);
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] = fmaf(x[r], A.scale2, bias[r] - lse2);
            } else {
                const float bias = (!BIAS ? 0.0f : hi <= A.far_lo ? table.lo : table.hi) - lse2;
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] = fmaf(x[r], A.scale2, bias);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) y[r] = exp2_fast(x[r]) * (y[r] - delta);
            if (j0 + TK > nwave_lo) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (j0 + block_row(r, g) >= nlane) y[r] = 0.0f;
            }
            if constexpr (BIAS) {
                if (near) {
                    near_bias(y, Ss + wave * 32 * kDiagPitch, Dg + wave * 64, j0 - (qw + shift), range, near_sum, lane);
                } else {
                    float s = 0.0f;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s += y[r];
                    if (hi <= A.far_lo) far_lo_sum += s;
                    else far_hi_sum += s;
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag ds = Ops<T>::from(y, s);
#pragma unroll
                for (int d = 0; d < DC / 32; ++d) Ops<T>::mma(dq[d], Kt::col_frag(K, 16 * s, 32 * d, lane), ds);
            }
        }
        if (t + 1 < tiles) {
            Kt::store(Ks[(t + 1) & 1], rk);
            Kt::store(Vs[(t + 1) & 1], rv);
        }
        __syncthreads();
    }
    if constexpr (BIAS) {
#pragma unroll
        for (int w = 1; w < 64; w *= 2) {
            far_lo_sum += __shfl_xor(far_lo_sum, w, 64);
            far_hi_sum += __shfl_xor(far_hi_sum, w, 64);
        }
        float* part = A.part + ((bh * A.qtiles + qt) * 4 + wave) * A.buckets;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int k = lane + 64 * n;
            if (k >= A.buckets) continue;
            float s = near_sum[n];
            if (k == A.far_lo_bucket) s += far_lo_sum;
            if (k == A.far_hi_bucket) s += far_hi_sum;
            as_global(part)[k] = s;
        }
    }
    if (i >= A.len_q) return;
    store_rows<T, DC>(at_row<T>(A.dq, b, i, h), dq, A.scale, A.dim, lane);
}

// rel[h][c] = bias[bucket(c)][h] log2(e), where c counts the offsets key -
// query from -(lq_pad - 1) on.
__global__ __launch_bounds__(NT) void attn_bias_kernel(AttnArgs A) {
    const int64_t c = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (c >= A.rel_ld) return;
    const int n = Bias::bucket_of(A.borders, (int)(c - (A.lq_pad - 1)) - (A.len_k - A.len_q));
    for (int h = 0; h < A.heads; ++h)
        as_global(A.rel)[h * A.rel_ld + c] = as_global(A.bias)[(int64_t)n * A.heads + h] * kLog2e;
}

// Calls f with the element type, the head width rounded up to 32 and whether there is a bias as constants.
template <typename F>
void by_form(bool bf16, int dim, bool bias, F f) {
    auto width = [&](auto t, auto b) {
        if (dim <= 32) f(t, std::integral_constant<int, 32>(), b);
        else if (dim <= 64) f(t, std::integral_constant<int, 64>(), b);
        else if (dim <= 96) f(t, std::integral_constant<int, 96>(), b);
        else f(t, std::integral_constant<int, 128>(), b);
    };
    auto type = [&](auto b) {
        if (bf16) width((__bf16*)nullptr, b);
        else width((float*)nullptr, b);
    };
    if (bias) type(std::true_type());
    else type(std::false_type());
}

template <typename T, int DC>
constexpr int key_blocks() {
    return 1;
}

}  // namespace

int attn_key_rows(bool bf16, int dim) {
    int n = 0;
    by_form(bf16, dim, false, [&](auto* t, auto dc, auto) {
        n = kAttnRows * key_blocks<std::remove_pointer_t<decltype(t)>, decltype(dc)::value>();
    });
    return n;
}

hipError_t launch_attn_bias(const AttnArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(attn_bias_kernel, dim3((unsigned)ceil_div(a.rel_ld, NT)), dim3(NT), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_attn_forward(const AttnArgs& a, bool bf16, hipStream_t stream) {
    by_form(bf16, a.dim, a.buckets != 0, [&](auto* t, auto dc, auto bias) {
        using T = std::remove_pointer_t<decltype(t)>;
        const dim3 grid((unsigned)((int64_t)a.batch * a.heads * a.qtiles));
        hipLaunchKernelGGL((attn_forward_kernel<T, decltype(dc)::value, decltype(bias)::value>), grid, dim3(NT), 0, stream,
                           a);
    });
    return hipGetLastError();
}

hipError_t launch_attn_dq(const AttnArgs& a, bool bf16, hipStream_t stream) {
    by_form(bf16, a.dim, a.buckets != 0, [&](auto* t, auto dc, auto bias) {
        using T = std::remove_pointer_t<decltype(t)>;
        const dim3 grid((unsigned)((int64_t)a.batch * a.heads * a.qtiles));
        hipLaunchKernelGGL((attn_dq_kernel<T, decltype(dc)::value, decltype(bias)::value>), grid, dim3(NT), 0, stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_attn_dkdv(const AttnArgs& a, bool bf16, hipStream_t stream) {
    by_form(bf16, a.dim, a.buckets != 0, [&](auto* t, auto dc, auto bias) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int DC = decltype(dc)::value;
        const int64_t tiles = (int64_t)a.batch * a.kv_heads * a.parts * a.ktiles;
        const dim3 grid((unsigned)(tiles + (int64_t)a.buckets * a.heads));
        if (grid.x != 0)
            hipLaunchKernelGGL((attn_dkdv_kernel<T, DC, key_blocks<T, DC>(), decltype(bias)::value>), grid, dim3(NT), 0,
                               stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_attn_kv_sum(const AttnArgs& a, bool bf16, hipStream_t stream) {
    const dim3 grid((unsigned)ceil_div((int64_t)a.batch * a.kv_heads * a.len_k * (a.dim / 8), NT), 2);
    if (bf16) hipLaunchKernelGGL(attn_kv_sum_kernel<__bf16>, grid, dim3(NT), 0, stream, a);
    else hipLaunchKernelGGL(attn_kv_sum_kernel<float>, grid, dim3(NT), 0, stream, a);
    return hipGetLastError();
}

}  // namespace kfac
