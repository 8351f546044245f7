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
#include <algorithm>
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
    // registers 8 s .. 8 s + 7 of a block, rounded to nearest even: the
    // probabilities and dS become operands of the type that the matrix cores
    // take.  Each term is off by at most 2^-8 of itself, as an input stored in
    // bfloat16 is; the sums over the terms are float32.
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
    using Frag = typename Ops<T>::Frag;

    static __device__ __forceinline__ int swz(int row) {
        if constexpr (CH == 4) return (row >> 2) & 3;
        else if constexpr (CH == 8) return (((row >> 1) & 1) << 2) | (((row >> 2) & 1) << 1) | ((row >> 3) & 1);
        else return ((row & 3) << 2) | ((row >> 2) & 3);
    }
    static __device__ __forceinline__ int at(int row, int chunk) { return row * PITCH + ((chunk ^ swz(row)) << 4); }

    // Copies from memory straight into LDS by THREADS threads (one wave, or
    // the workgroup), 16 bytes each: a wave's copies land one after another,
    // so the chunks' permutation is taken on the memory side.
    template <int THREADS>
    struct Feed {
        static constexpr int ALL = ROWS * CH, COPIES = ALL < THREADS ? 1 : ALL / THREADS;
        static_assert(ALL % 64 == 0 && (ALL < THREADS || ALL % THREADS == 0), "whole waves of copies");
        uint32_t off[COPIES];
        int stride, row_bytes, wave;
        __device__ __forceinline__ Feed(int thread, int64_t stride_elements, int dim)
            : stride((int)stride_elements * ES), row_bytes(dim * ES),
              wave(__builtin_amdgcn_readfirstlane(thread >> 6)) {
#pragma unroll
            for (int n = 0; n < COPIES; ++n) {
                const int q = (wave * COPIES + n) * 64 + (thread & 63), row = q / CH, chunk = (q % CH) ^ swz(row);
                off[n] = chunk * 16 < row_bytes ? (uint32_t)(row * stride + chunk * 16) : kOOB;
            }
        }
        // the tile at `base`, of which `rows` rows exist (the others read as zero)
        __device__ __forceinline__ void operator()(char* lds, const char* base, int rows) const {
            const int n = min(rows, ROWS);
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<char*>(base), (short)0, n > 0 ? (n - 1) * stride + row_bytes : 0, 0x00020000);
            if (ALL < THREADS && wave * 64 >= ALL) return;
#pragma unroll
            for (int n = 0; n < COPIES; ++n)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rs, (__attribute__((address_space(3))) void*)(lds + (wave * COPIES + n) * 1024), 16, off[n], 0, 0, 0);
        }
    };
    // A lane's places in any tile of this form.  The permutation is an
    // exclusive or, so a fragment's address is its lane's place with a few
    // constant bits turned over; fresh() keeps the compiler from holding
    // every such address in a register of its own over the loop.
    struct Lane {
        int row, col, own;
        __device__ __forceinline__ explicit Lane(int lane) : own(lane) {
            const int g = lane >> 5, gr = lane >> 4, p = lane & 15;
            row = at(lane & 31, ES == 2 ? g : 2 * g);
            col = at(4 * (gr >> 1) + (p >> 2), 2 * (gr & 1) + ((p & 3) >> 1)) + (p & 1) * 8;   // bf16 only
        }
        __device__ __forceinline__ Lane fresh() const {
            Lane l = *this;
            asm volatile("" : "+v"(l.row), "+v"(l.col));
            return l;
        }
    };
    // Rows row0 + lane % 32 (row0 a multiple of 32), columns 16 s + 8 (lane / 32) .. + 7.
    static __device__ __forceinline__ Frag row_frag(const char* lds, int row0, int s, const Lane& l) {
        if constexpr (ES == 2) {
            return *reinterpret_cast<const bf16x8*>(lds + row0 * PITCH + (l.row ^ (s << 5)));
        } else {
            const floatx4 a = *reinterpret_cast<const floatx4*>(lds + row0 * PITCH + (l.row ^ (s << 6)));
            const floatx4 b = *reinterpret_cast<const floatx4*>(lds + row0 * PITCH + (l.row ^ (s << 6) ^ 16));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // Column 32 d + lane % 32, rows row0 + 4 g .. + 3 and row0 + 8 + 4 g .. + 3 (g = lane / 32, row0 a multiple of 16).
    static __device__ __forceinline__ Frag col_frag(const char* lds, int row0, int d, const Lane& l) {
        if constexpr (ES == 2) {
            constexpr int NEXT = CH == 8 ? 16 : 32;    // eight rows on: one bit of the chunk's number changes
            auto rd = [&](int at) {
                return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) short4v*)const_cast<char*>(lds + row0 * PITCH + at));
            };
            return __builtin_bit_cast(bf16x8,
                                      __builtin_shufflevector(rd(l.col ^ (d << 6)), rd((l.col ^ (d << 6) ^ NEXT) + 8 * PITCH),
                                                              0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int col = 32 * d + (l.own & 31), row = row0 + 4 * (l.own >> 5);
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

// 64 floats from memory (or zeros) into LDS, by one wave.
__device__ __forceinline__ void copy_stats(float* lds, const float* p, bool there, int lane) {
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p), (short)0, there ? 256 : 0, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)lds, 4, lane * 4, 0, 0,
                                             0);
}

// Until this wave's copies into LDS have arrived.
__device__ __forceinline__ void wait_copies() {
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
    asm volatile("" ::: "memory");
}

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

    // (`ids`: the offsets' buckets beside their bias)
    __device__ __forceinline__ void begin(const AttnArgs& A, float* table, int h, uint8_t* ids = nullptr) {
        near = table;
        rel = A.near_n ? nullptr : A.rel + h * A.rel_ld + (A.lq_pad - 1);
        lo = as_global(A.bias)[(int64_t)A.far_lo_bucket * A.heads + h] * kLog2e;
        hi = as_global(A.bias)[(int64_t)A.far_hi_bucket * A.heads + h] * kLog2e;
        for (int c = threadIdx.x; c < A.near_n; c += NT) {
            const int n = bucket_of(A.borders, A.far_lo - kAttnPad + c);
            table[c] = as_global(A.bias)[(int64_t)n * A.heads + h] * kLog2e;
            if (ids) ids[c] = (uint8_t)n;
        }
    }
    // (two values to choose from, not two places: the struct stays in registers)
    __device__ __forceinline__ float beyond(bool low) const {
        const float a = lo, b = hi;
        return low ? a : b;
    }
    static __device__ __forceinline__ int bucket_of(const AttnBorders& B, int d) {
        const int dist = B.two_sided ? abs(d) : max(-d, 0);
        int n = B.two_sided && d > 0 ? B.n + 1 : 0;
        // eight borders per load; what fills up the last eight lies beyond every distance
        for (int k = 0; k < B.n; k += 8)
#pragma unroll
            for (int u = 0; u < 8; ++u) n += dist >= B.at[k + u];
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

// Joins the sums of a deep workgroup's waves, each times its lane's `f`, in
// the order of the waves, and writes the rows: wave d writes columns 32 d ..,
// half of the blocks through either LDS buffer (16 KB per 32 columns).
template <typename T, int DC, typename Row>
__device__ __forceinline__ void join_waves(const floatx16 (&acc)[DC / 32], float f, float* X, float* Y, int wave, int lane,
                                           bool real, int dim, Row row) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < DC / 32; ++d) {
        float* p = (d & 1 ? Y : X) + ((d >> 1) * 4 + wave) * 1024;
#pragma unroll
        for (int r = 0; r < 16; ++r) p[64 * r + lane] = acc[d][r] * f;
    }
    __syncthreads();
    if (wave >= DC / 32 || !real) return;
    const float* p = (wave & 1 ? Y : X) + (wave >> 1) * 4096;
    floatx16 sum[1];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        float s = p[64 * r + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) s += p[1024 * w + 64 * r + lane];
        sum[0][r] = s;
    }
    store_rows<T, 32>(row() + 32 * wave * (int)sizeof(T), sum, 1.0f, dim - 32 * wave, lane);
}

// Item of a workgroup: in turns (blockIdx.y) of at least eight key and value
// heads, each turn in one contiguous range per XCD, so that a head's keys stay
// under one L2 and sequences of uneven length, which follow each other in the
// items' order, are dealt out over all XCDs.  With one turn, lengths from 0 to
// 2048 in 8 sequences (16 heads of 64, bfloat16) leave one XCD with a quarter
// of the work: the pass by queries takes 287 us instead of 195, the pass by
// keys 318 instead of 235.
__device__ __forceinline__ uint32_t turn_item() {
    return blockIdx.y * gridDim.x + (uint32_t)xcd_remap(blockIdx.x, gridDim.x);
}

// The workgroup's share of a pass by queries.  Wide: 128 queries, 32 per
// wave, and key tiles that all waves read.  Deep (few queries in all): 32
// queries, and every wave takes every fourth tile of 32 keys, through LDS of
// its own and at its own pace; the waves' sums are joined at the end.
template <bool DEEP>
struct QueryShare {
    int b, h, hk, qt, qw, i, nk, shift, nwg, nlane, nwave_lo, nwave_hi;
    int64_t bh;
    __device__ __forceinline__ QueryShare(const AttnArgs& A, int wave, int lane) {
        const uint32_t item = turn_item();
        bh = item / (uint32_t)A.qtiles;
        qt = A.qtiles - 1 - (int)(item % (uint32_t)A.qtiles);   // the longest rows of a causal head first
        b = (int)((uint32_t)bh / (uint32_t)A.heads);
        h = (int)((uint32_t)bh % (uint32_t)A.heads);
        hk = h / A.group;
        shift = A.len_k - A.len_q;
        const int rows = DEEP ? 32 : kAttnRows, q0 = qt * rows;
        qw = DEEP ? q0 : q0 + 32 * wave;
        i = qw + (lane & 31);
        nk = visible_keys(A, b);
        // keys this workgroup, this lane's query and this wave's first and last query may see
        const int last = min(A.len_q, q0 + rows) - 1;
        nwg = A.causal ? max(0, min(nk, last + shift + 1)) : nk;
        nlane = A.causal ? max(0, min(nk, i + shift + 1)) : nk;
        nwave_lo = A.causal ? max(0, min(nk, qw + shift + 1)) : nk;
        nwave_hi = qw >= A.len_q ? 0 : A.causal ? max(0, min(nk, qw + 31 + shift + 1)) : nk;
    }
};

// LDS of a pass by queries: key and value tiles, two of each where they fit
// beside what else the kernel keeps.
template <typename T, int DC, bool DEEP, int ROWS>
struct KeyTiles {
    using Kt = Tile<T, DC, ROWS>;
    static constexpr int WAVES = DEEP ? 4 : 1;
    static constexpr int BUFS = DEEP && Kt::PITCH >= 256 ? 1 : 2;
    static constexpr int BYTES = WAVES * Kt::BYTES;
    // the first buffer of a deep pass also joins the waves' sums
    static constexpr int FIRST = DEEP && BYTES < 16384 ? 16384 : BYTES;
    static_assert(!DEEP || (BYTES >= (DC / 32) / 2 * 16384 && FIRST >= (DC / 32 + 1) / 2 * 16384), "room for the join");
};

// Runs body(K, V, first key) over the key tiles.  The copies of the next
// tile run beside the products of this one.
template <typename T, int DC, bool DEEP, int ROWS, typename Body>
__device__ __forceinline__ void over_keys(const AttnArgs& A, const QueryShare<DEEP>& S, char* K0, char* K1, char* V0,
                                          char* V1, int wave, Body body) {
    using L = KeyTiles<T, DC, DEEP, ROWS>;
    using Kt = typename L::Kt;
    constexpr int THREADS = DEEP ? 64 : NT, STEP = DEEP ? 4 * ROWS : ROWS;
    const int own = DEEP ? wave * Kt::BYTES : 0;
    const typename Kt::template Feed<THREADS> fk(threadIdx.x & (THREADS - 1), A.k.sl, A.dim),
        fv(threadIdx.x & (THREADS - 1), A.v.sl, A.dim);
    int j = DEEP ? wave * ROWS : 0;
    const char *kp = at_row<T>(A.k, S.b, j, S.hk), *vp = at_row<T>(A.v, S.b, j, S.hk);
    const int64_t ks = A.k.sl * (int64_t)sizeof(T) * STEP, vs = A.v.sl * (int64_t)sizeof(T) * STEP;
    int next = j;
    auto fetch = [&](char* K, char* V) {
        if (next >= S.nwg) return;
        fk(K + own, kp, S.nk - next);
        fv(V + own, vp, S.nk - next);
        kp += ks;
        vp += vs;
        next += STEP;
    };
    auto arrive = [&]() {
        wait_copies();
        if (!DEEP) __syncthreads();
    };
    fetch(K0, V0);
    arrive();
    if constexpr (L::BUFS == 2) {
        while (j < S.nwg) {
            fetch(K1, V1);
            body(K0 + own, V0 + own, j);
            arrive();
            j += STEP;
            // (past the last tile the body does nothing; leaving here
            // instead would give every sum two places to live)
            fetch(K0, V0);
            body(K1 + own, V1 + own, j);
            arrive();
            j += STEP;
        }
    } else {
        while (j < S.nwg) {
            body(K0 + own, V0 + own, j);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // every read of the tile is done
            fetch(K0, V0);
            arrive();
            j += STEP;
        }
    }
}

// ---------------------------------------------------------------- forward --
// The running maximum is raised only when a score exceeds it by more than
// kSlack (log2 units): until then the probabilities stay below 2^kSlack, the
// sums below 2^kSlack times the number of keys, and nothing is rescaled (8192
// causal rows, heads of 128: 330 us, raised at every new maximum 348).
constexpr float kSlack = 8.0f;

// out and lse.  A tile of 64 keys (32 in float32 and in deep workgroups) lies
// in LDS for the workgroup's four waves; queries, scores and sums stay in
// registers.  8192 causal rows, 16 heads of 128 over 4 of keys, bfloat16:
// 328 us, 838 TFLOP/s of the 1283 of a large library product; the matrix
// cores are busy 33 % of the time at their peak rate, the exponentials and
// conversions (about 200 vector instructions per 32 x 32 block) take most of
// the rest of the issue slots.  8 sequences of up to 512, 16 heads of 64:
// 19 us, bound by the latency of one wave's chain of steps (1.1 us per tile).
template <typename T, int DC, bool BIAS, bool DEEP>
__global__ __launch_bounds__(NT, sizeof(T) == 2 || DC <= 64 ? 2 : 1) void attn_forward_kernel(AttnArgs A) {
    constexpr int TK = sizeof(T) == 2 && !DEEP ? 64 : 32;
    using L = KeyTiles<T, DC, DEEP, TK>;
    using Kt = typename L::Kt;
    __shared__ __attribute__((aligned(16))) char K0[L::FIRST];
    __shared__ __attribute__((aligned(16))) char V0[L::BYTES];
    __shared__ __attribute__((aligned(16))) char K1[L::BUFS == 2 ? L::BYTES : 16];
    __shared__ __attribute__((aligned(16))) char V1[L::BUFS == 2 ? L::BYTES : 16];
    __shared__ float Near[BIAS ? kAttnNear : 1];
    using Frag = typename Ops<T>::Frag;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), g = lane >> 5;
    const QueryShare<DEEP> S(A, wave, lane);

    Frag qf[DC / 16];
    own_frags<T, DC>(qf, at_row<T>(A.q, S.b, S.qw, S.h), A.q.sl * (int64_t)sizeof(T), lane & 31, A.len_q - S.qw, A.dim,
                     lane);
    Bias table;
    if constexpr (BIAS) {
        table.begin(A, Near, S.h);
        if constexpr (DEEP) __syncthreads();
    }
    floatx16 o[DC / 32];
    clear(o);
    const typename Kt::Lane place(lane);
    float m = -INFINITY, l = 0.0f;   // the base of this lane's query and its own half of the sum
    over_keys<T, DC, DEEP, TK>(A, S, K0, K1, V0, V1, wave, [&](const char* K, const char* V, int j0) {
        if (j0 >= S.nwave_hi) return;
        const typename Kt::Lane& pl = place;
        floatx16 x[TK / 32];
        clear(x);
#pragma unroll
        for (int u = 0; u < TK / 32; ++u)
#pragma unroll
            for (int s = 0; s < DC / 16; ++s) Ops<T>::mma(x[u], Kt::row_frag(K, 32 * u, s, pl), qf[s]);
        // scores in log2 units are x scale2 + shift
        const int lo = j0 - (S.qw + 31 + S.shift), hi = j0 + TK - 1 - (S.qw + S.shift);
        float scale2 = A.scale2, shift = 0.0f;
        if constexpr (BIAS) {
            if (lo >= A.far_hi || hi <= A.far_lo) {
                shift = table.beyond(hi <= A.far_lo);
            } else {
#pragma unroll
                for (int u = 0; u < TK / 32; ++u) {
                    floatx16 bias;
                    table.block<true>(bias, A, j0 + 32 * u, S.i, g);
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[u][r] = fmaf(x[u][r], A.scale2, bias[r]);
                }
                scale2 = 1.0f;
            }
        }
        if (j0 + TK > S.nwave_lo) {
#pragma unroll
            for (int u = 0; u < TK / 32; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    x[u][r] = j0 + 32 * u + block_row(r, g) >= S.nlane ? -INFINITY : x[u][r];
        }
        float top = x[0][0];
#pragma unroll
        for (int u = 0; u < TK / 32; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, x[u][r]);
        top = fmaxf(top, other_half(top));
        top = fmaf(top, scale2, shift);
        if (__any(top > m + kSlack)) {
            // raise the base: each lane to its own maximum (one that has seen nothing keeps -inf and 0)
            const float up = fmaxf(m, top), keep = up == -INFINITY ? 0.0f : exp2_fast(m - up);
            m = up;
            l *= keep;
#pragma unroll
            for (int d = 0; d < DC / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[d][r] *= keep;
        }
        shift -= m == -INFINITY ? 0.0f : m;
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < TK / 32; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                x[u][r] = exp2_fast(fmaf(x[u][r], scale2, shift));
                sum += x[u][r];
            }
        l += sum;
#pragma unroll
        for (int u = 0; u < TK / 32; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag p = Ops<T>::from(x[u], s);
#pragma unroll
                for (int d = 0; d < DC / 32; ++d) Ops<T>::mma(o[d], Kt::col_frag(V, 32 * u + 16 * s, d, pl), p);
            }
    });
    l += other_half(l);
    const bool real = S.i < A.len_q;
    if constexpr (!DEEP) {
        if (!real) return;
        store_rows<T, DC>(at_row<T>(A.out, S.b, S.i, S.h), o, l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l, A.dim, lane);
        if (g == 0) as_global(A.lse)[S.bh * A.len_q + S.i] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
    } else {
        // the waves' bases and sums, then their outputs at the common base
        __shared__ float Ms[2][4][32];
        if (g == 0) {
            Ms[0][wave][lane] = m;
            Ms[1][wave][lane] = l;
        }
        __syncthreads();
        float top = -INFINITY, total = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, Ms[0][w][lane & 31]);
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int w = 0; w < 4; ++w) total = fmaf(Ms[1][w][lane & 31], exp2_fast(Ms[0][w][lane & 31] - base), total);
        const float f = exp2_fast(m - base) * (total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total);
        join_waves<T, DC>(o, f, reinterpret_cast<float*>(K0), reinterpret_cast<float*>(V0), wave, lane, real, A.dim,
                          [&]() { return at_row<T>(A.out, S.b, S.i, S.h); });
        if (wave == 0 && g == 0 && real)
            as_global(A.lse)[S.bh * A.len_q + S.i] = total == 0.0f ? -INFINITY : fmaf(top, kLn2, logf(total));
    }
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

// dK and dV of 128 keys, 32 per wave; queries pass by in tiles of 32 QB:
// those of one query head of the group and one chunk of its rows where the
// key tiles are shared out in parts (`parts` > 1, the shares summed by
// attn_kv_sum_kernel), else all.  The workgroups past the key tiles sum the
// bias gradient.  Four products per 32 x 32 block.  8192 causal rows, 16 heads
// of 128 over 4 of keys, bfloat16: 540 to 575 us, 960 to 1020 TFLOP/s of the
// 1283 of a large library product: LDS reads of the two tiles by rows and by
// columns and the matrix cores take about the same time.  8 sequences of up to
// 512, 16 heads of 64: 28.5 us, bound by latency (1.8 us per step of 64
// queries, 4.5 us before the first, 2 us after the last); 333 x 401 in
// float32, 18 heads of 72: 42 us.
template <typename T, int DC, int QB, bool BIAS>
__device__ __forceinline__ void dkdv_item(const AttnArgs& A) {
    constexpr int TQ = 32 * QB;
    using Qt = Tile<T, DC, TQ>;
    __shared__ __attribute__((aligned(16))) char Q0[Qt::BYTES];
    __shared__ __attribute__((aligned(16))) char Q1[Qt::BYTES];
    __shared__ __attribute__((aligned(16))) char D0[Qt::BYTES];
    __shared__ __attribute__((aligned(16))) char D1[Qt::BYTES];
    __shared__ __attribute__((aligned(16))) float L0[2 * TQ];
    __shared__ __attribute__((aligned(16))) float L1[2 * TQ];
    __shared__ float Near[BIAS ? kAttnNear : NT];
    // wide bf16 heads: the values stay in LDS instead of registers, which
    // leaves room for two waves per SIMD (8192 causal, heads of 128: 538 us
    // instead of 753)
    constexpr bool VLDS = sizeof(T) == 2 && DC > 64;
    using Vt = Tile<T, DC, kAttnRows>;
    __shared__ __attribute__((aligned(16))) char Vs[VLDS ? Vt::BYTES : 16];
    using Frag = typename Ops<T>::Frag;
    // key tiles fastest: neighbours read the same queries
    const uint32_t item = turn_item(), tiles = (uint32_t)A.batch * A.kv_heads * A.parts * A.ktiles;
    if (item >= tiles) {
        if (BIAS && item - tiles < (uint32_t)(A.buckets * A.heads)) sum_bias(A, Near, (int)(item - tiles));
        return;
    }
    const int kt = (int)(item % (uint32_t)A.ktiles);
    const uint32_t rest = item / (uint32_t)A.ktiles;
    const int part = (int)(rest % (uint32_t)A.parts);
    const uint32_t bk = rest / (uint32_t)A.parts;
    const int b = (int)(bk / (uint32_t)A.kv_heads), hk = (int)(bk % (uint32_t)A.kv_heads);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), g = lane >> 5;
    const int shift = A.len_k - A.len_q;
    const int k0 = kt * kAttnRows, kw = k0 + 32 * wave, j = kw + (lane & 31);
    const int nk = visible_keys(A, b);

    Frag kf[DC / 16], vf[VLDS ? 1 : DC / 16];
    floatx16 dk[DC / 32], dv[DC / 32];
    own_frags<T, DC>(kf, at_row<T>(A.k, b, kw, hk), A.k.sl * (int64_t)sizeof(T), lane & 31, nk - kw, A.dim, lane);
    if constexpr (!VLDS)
        own_frags<T, DC>(vf, at_row<T>(A.v, b, kw, hk), A.v.sl * (int64_t)sizeof(T), lane & 31, nk - kw, A.dim, lane);
    clear(dk);
    clear(dv);

    // query tiles of this part, from the first one that sees key k0 (causal: j <= i + shift)
    const int heads = A.parts > 1 ? 1 : A.group, chunks = A.parts > 1 ? A.parts / A.group : 1;
    const int h0 = hk * A.group + (A.parts > 1 ? part / chunks : 0);
    const int qtiles = (A.len_q + TQ - 1) / TQ;
    const int first = max(A.causal ? max(0, k0 - shift) / TQ : 0, part % chunks * A.qchunk);
    const int per = k0 < nk ? max(0, min(qtiles, (part % chunks + 1) * A.qchunk) - first) : 0;
    const int steps = per * heads;
    const int end = min(A.len_q, (first + per) * TQ);   // queries of this part
    Bias table;
    const typename Qt::template Feed<NT> fq(threadIdx.x, A.q.sl, A.dim), fd(threadIdx.x, A.dout.sl, A.dim);
    const char *qp = nullptr, *dp = nullptr;
    const float* sp = nullptr;
    int fh = h0, fi = 0, fetched = 0;      // head and query tile of the next fetch
    // (past the last tile: zeros, which the body hides)
    auto fetch = [&](char* Q, char* D, float* L) {
        if (fi == 0) {
            qp = at_row<T>(A.q, b, first * TQ, fh);
            dp = at_row<T>(A.dout, b, first * TQ, fh);
            sp = A.stats + (((int64_t)b * A.heads + fh) * A.lq_pad + first * TQ) * 2;
        }
        const int left = fetched < steps ? A.len_q - (first + fi) * TQ : 0;
        fq(Q, qp, left);
        fd(D, dp, left);
        // (32 queries' numbers per wave; those past the last query are not there)
        if (wave < QB) copy_stats(L + 64 * wave, sp + 64 * wave, left > 32 * wave, lane);
        qp += A.q.sl * (int64_t)sizeof(T) * TQ;
        dp += A.dout.sl * (int64_t)sizeof(T) * TQ;
        sp += 2 * TQ;
        ++fetched;
        if (++fi == per) {
            fi = 0;
            ++fh;
        }
    };
    int h = h0, i0 = first * TQ;
    const typename Qt::Lane place(lane);
    auto body = [&](const char* Q, const char* D, const float* L) {
        // (A wave whose keys are all hidden from these queries adds zeros: a
        // branch around the sums would cost every wave their copies.)
        const typename Qt::Lane pl = place.fresh();
        typename Vt::Lane pv(0);
        pv.row = pl.row;
        // x = q k - lse / scale2 and y = dout v - delta, row by row (-inf, 0
        // where a row sees nothing).  The bfloat16 sums begin with the rows'
        // numbers; the float32 ones take them at the end, since a sum that
        // begins with a large number rounds every product to it.
        constexpr bool FIRST = sizeof(T) == 2;
        floatx16 x[QB], y[QB];
        auto rows = [&](auto f) {
#pragma unroll
            for (int u = 0; u < QB; ++u)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const floatx4 l4 = *reinterpret_cast<const floatx4*>(L + 64 * u + 8 * t + 4 * g);
                    const floatx4 e4 = *reinterpret_cast<const floatx4*>(L + 64 * u + 32 + 8 * t + 4 * g);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        x[u][4 * t + c] = f(x[u][4 * t + c], l4[c]);
                        y[u][4 * t + c] = f(y[u][4 * t + c], e4[c]);
                    }
                }
        };
        if constexpr (FIRST) {
            rows([](float, float number) { return number; });
        } else {
            clear(x);
            clear(y);
        }
#pragma unroll
        for (int s = 0; s < DC / 16; ++s)
#pragma unroll
            for (int u = 0; u < QB; ++u) Ops<T>::mma(x[u], Qt::row_frag(Q, 32 * u, s, pl), kf[s]);
        if constexpr (QB == 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < DC / 16; ++s)
#pragma unroll
            for (int u = 0; u < QB; ++u) {
                const Frag f = Qt::row_frag(D, 32 * u, s, pl);
                if constexpr (VLDS) Ops<T>::mma(y[u], f, Vt::row_frag(Vs, 32 * wave, s, pv));
                else Ops<T>::mma(y[u], f, vf[s]);
            }
        if constexpr (!FIRST)
            rows([](float sum, float number) { return sum + number; });
        if constexpr (QB == 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < QB; ++u) {
            const int iu = i0 + 32 * u;
            // The second body of an odd count of steps, and the last of a
            // step's blocks, may lie past the queries: their offsets are in
            // no table, and their numbers (zeros, and where rows repeat the
            // last row's values) would give exp(bias) as probabilities, so
            // every key is hidden from them.  Rows past the last query in a
            // block that has some get probability 0 from their lse.
            const bool there = iu < end;
            float far = 0.0f;
            bool near = false;
            if constexpr (BIAS) {
                const int lo = kw - (iu + 31 + shift), hi = kw + 31 - (iu + shift);
                near = there && !(lo >= A.far_hi || hi <= A.far_lo);
                far = table.beyond(hi <= A.far_lo);
            }
            if (BIAS && near) {
                floatx16 bias;
                table.block<false>(bias, A, iu, j, g);
#pragma unroll
                for (int r = 0; r < 16; ++r) x[u][r] = exp2_fast(fmaf(x[u][r], A.scale2, bias[r]));
            } else {
#pragma unroll
                for (int r = 0; r < 16; ++r) x[u][r] = exp2_fast(fmaf(x[u][r], A.scale2, far));
            }
            if (!there | (kw + 32 > nk) | (A.causal & (kw + 31 > iu + shift))) {
                // this key is hidden from the block's first `hidden` rows
                const int hidden = !there | (j >= nk) ? 32 : A.causal ? j - iu - shift : 0;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const bool hide = block_row(r, g) < hidden;
                    x[u][r] = hide ? 0.0f : x[u][r];
                    y[u][r] = hide ? 0.0f : y[u][r];
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) y[u][r] *= x[u][r];
        }
        if constexpr (QB == 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < QB; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag p = Ops<T>::from(x[u], s), ds = Ops<T>::from(y[u], s);
#pragma unroll
                for (int d = 0; d < DC / 32; ++d) {
                    Ops<T>::mma(dv[d], Qt::col_frag(D, 32 * u + 16 * s, d, pl), p);
                    Ops<T>::mma(dk[d], Qt::col_frag(Q, 32 * u + 16 * s, d, pl), ds);
                }
            }
    };
    auto advance = [&](bool more) {
        wait_copies();
        i0 += TQ;
        if (i0 >= (first + per) * TQ && more) {
            i0 = first * TQ;
            ++h;
            if constexpr (BIAS) {
                __syncthreads();           // every wave is done with the last head's table
                table.begin(A, Near, h);
            }
        }
        __syncthreads();
    };
    if (steps > 0) {
        if constexpr (VLDS) {
            const typename Vt::template Feed<NT> fv(threadIdx.x, A.v.sl, A.dim);
            fv(Vs, at_row<T>(A.v, b, k0, hk), nk - k0);
        }
        fetch(Q0, D0, L0);
        if constexpr (BIAS) table.begin(A, Near, h);
        wait_copies();
    }
    __syncthreads();
    for (int st = 0; st < steps; st += 2) {
        fetch(Q1, D1, L1);
        body(Q0, D0, L0);
        advance(st + 1 < steps);
        fetch(Q0, D0, L0);
        body(Q1, D1, L1);
        advance(st + 2 < steps);
    }
    if (j >= A.len_k) return;
    if (A.parts > 1) {
        const int64_t row = ((int64_t)part * A.batch * A.kv_heads + (int64_t)bk) * A.len_k + j;
        const int64_t all = (int64_t)A.parts * A.batch * A.kv_heads * A.len_k;
        store_rows<float, DC>(reinterpret_cast<char*>(A.kv_part + row * A.dim), dk, A.scale, A.dim, lane);
        store_rows<float, DC>(reinterpret_cast<char*>(A.kv_part + (all + row) * A.dim), dv, 1.0f, A.dim, lane);
    } else {
        store_rows<T, DC>(at_row<T>(A.dk, b, j, hk), dk, A.scale, A.dim, lane);
        store_rows<T, DC>(at_row<T>(A.dv, b, j, hk), dv, 1.0f, A.dim, lane);
    }
}

template <typename T, int DC, int QB, bool BIAS>
__global__ __launch_bounds__(NT, sizeof(T) == 2 ? 2 : 1) void attn_dkdv_kernel(AttnArgs A) {
    dkdv_item<T, DC, QB, BIAS>(A);
}

// dk (blockIdx.y = 0) and dv from their shares, in the shares' order; eight
// values per thread.  4 shares of 8192 x 4 heads of 128: 134 MB read in 22 us,
// 6.1 TB/s with what the caches still hold.
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
// queries) that spans several buckets: the block goes through LDS, lanes t and
// t + 32 sum the diagonals key - query = t - 32 and t, which have 32 elements
// together, each lane half of the rows, so that lane t has diagonal t - 32.  A
// scan over the lanes sums each bucket's run of diagonals up to its last lane,
// and lane n takes that sum for buckets n and n + 64.  One lane per diagonal
// reads twice as much: 8192 causal rows 485 us instead of 455.  (Adding a bucket's diagonals one after another,
// each an LDS read behind the last, took most of the pass; plain prefix sums
// and their differences would round a small bucket to its neighbours' size.)
// `base` is the offset of the block's diagonal 0, `id` the bucket of this
// lane's diagonal.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// Adds the sum of the lane that CTRL names where it is of the same bucket.
template <int CTRL, int ROWS>
__device__ __forceinline__ void add_run(float& v, int id) {
    const float from = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
    const int same = __builtin_amdgcn_update_dpp(-1, id, CTRL, ROWS, 0xf, false);
    v += same == id ? from : 0.0f;
}
// Sum of v over the lanes up to this one that have its id (ids stand in runs).
__device__ __forceinline__ float run_sum(float v, int id) {
    add_run<0x111, 0xf>(v, id);   // within rows of 16 lanes: 1, 2, 4 and 8 lanes up
    add_run<0x112, 0xf>(v, id);
    add_run<0x114, 0xf>(v, id);
    add_run<0x118, 0xf>(v, id);
    add_run<0x142, 0xa>(v, id);   // the last lane of rows 0 and 2 to rows 1 and 3
    add_run<0x143, 0xc>(v, id);   // lane 31 to the upper half
    return v;
}
constexpr int kDiagPitch = 33;
__device__ __forceinline__ void near_bias(const floatx16& ds, float* S, float* diag, int base, int id,
                                          const int2 (&range)[2], float (&sum)[2], int lane) {
    const int g = lane >> 5;
    // (a number of which the compiler cannot keep sixteen comparisons over the loop)
    const int t = lane & 31;
    int beyond = 16 * g - t;
    asm volatile("" : "+v"(beyond));
#pragma unroll
    for (int r = 0; r < 16; ++r) S[block_row(r, g) * kDiagPitch + t] = ds[r];
    wave_fence();
    float up = 0.0f, down = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int row = 16 * g + r;
        const float v = S[row * kDiagPitch + ((row - t) & 31)];
        up += beyond >= -r ? v : 0.0f;
        down += beyond >= -r ? 0.0f : v;
    }
    const float d = (g ? up : down) + other_half(g ? down : up);
    diag[lane] = run_sum(d, id);
    wave_fence();
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        // diagonals lo .. hi of the block's 63, none where hi < lo
        const int lo = max(range[n].x - base, -31), hi = min(range[n].y - base, 31);
        const float run = diag[max(0, hi + 32)];
        sum[n] += hi < lo ? 0.0f : run;
    }
    wave_fence();
}

// dQ and the waves' shares of the bias gradient.  Three products per 32 x 32
// block, of which two are the scores and dP again.  8192 causal rows, 16 heads
// of 128 over 4 of keys, bfloat16: 455 to 470 us, 880 to 906 TFLOP/s of the 1283
// of a large library product, bound by vector instructions; 8 sequences of up to
// 512, 16 heads of 64: 29 us (0.7 us per block of 32 keys, twice that where the bias
// is near); 333 x 401 in float32, 18 heads of 72: 32 us.  Leaves -lse / scale2 and
// -delta of every query for the pass by keys.
template <typename T, int DC, bool BIAS, bool DEEP>
__global__ __launch_bounds__(NT, sizeof(T) == 2 && !(BIAS && DEEP && DC > 32) ? 2 : 1) void attn_dq_kernel(AttnArgs A) {
    constexpr int TK = 32;
    using L = KeyTiles<T, DC, DEEP, TK>;
    using Kt = typename L::Kt;
    __shared__ __attribute__((aligned(16))) char K0[L::FIRST];
    __shared__ __attribute__((aligned(16))) char V0[L::BYTES];
    __shared__ __attribute__((aligned(16))) char K1[L::BUFS == 2 ? L::BYTES : 16];
    __shared__ __attribute__((aligned(16))) char V1[L::BUFS == 2 ? L::BYTES : 16];
    __shared__ float Ss[BIAS ? 4 * 32 * kDiagPitch : 1];
    __shared__ float Dg[BIAS ? 4 * 64 : 1];
    __shared__ float Near[BIAS ? kAttnNear : 1];
    __shared__ uint8_t Ids[BIAS ? kAttnNear : 1];
    using Frag = typename Ops<T>::Frag;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), g = lane >> 5;
    const QueryShare<DEEP> S(A, wave, lane);
    const int i = S.i;

    Frag qf[DC / 16], df[DC / 16];
    own_frags<T, DC>(qf, at_row<T>(A.q, S.b, S.qw, S.h), A.q.sl * (int64_t)sizeof(T), lane & 31, A.len_q - S.qw, A.dim,
                     lane);
    own_frags<T, DC>(df, at_row<T>(A.dout, S.b, S.qw, S.h), A.dout.sl * (int64_t)sizeof(T), lane & 31, A.len_q - S.qw,
                     A.dim, lane);
    // delta from the rows in registers, and lse in log2 units.  Rows that see
    // nothing, and rows past the last, get lse = +inf: every probability 0.
    float lse2 = INFINITY, delta = 0.0f;
    {
        Frag of[DC / 16];
        own_frags<T, DC>(of, at_row<T>(A.out, S.b, S.qw, S.h), A.out.sl * (int64_t)sizeof(T), lane & 31, A.len_q - S.qw,
                         A.dim, lane);
#pragma unroll
        for (int s = 0; s < DC / 16; ++s)
#pragma unroll
            for (int t = 0; t < 8; ++t) delta = fmaf((float)df[s][t], (float)of[s][t], delta);
        delta += other_half(delta);
        if (i < A.len_q) {
            const float v = as_global(A.lse)[S.bh * A.len_q + i];
            if (v != -INFINITY) lse2 = v * kLog2e;
        }
        // [32 queries][lse, delta]: lane half g writes its kind
        if (!DEEP || wave == 0)
            as_global(A.stats)[(S.bh * A.lq_pad + S.qw) * 2 + lane] = g == 0 ? -lse2 / A.scale2 : -delta;
    }
    Bias table;
    float near_sum[2] = {0.0f, 0.0f}, far_lo_sum = 0.0f, far_hi_sum = 0.0f;
    int2 range[2];
    if constexpr (BIAS) {
        table.begin(A, Near, S.h, Ids);
        if constexpr (DEEP) __syncthreads();
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
    const typename Kt::Lane place(lane);
    over_keys<T, DC, DEEP, TK>(A, S, K0, K1, V0, V1, wave, [&](const char* K, const char* V, int j0) {
        if (j0 >= S.nwave_hi) return;
        const typename Kt::Lane pl = place.fresh();
        floatx16 x, y;
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.0f;
#pragma unroll
        for (int s = 0; s < DC / 16; ++s) Ops<T>::mma(x, Kt::row_frag(K, 0, s, pl), qf[s]);
#pragma unroll
        for (int s = 0; s < DC / 16; ++s) Ops<T>::mma(y, Kt::row_frag(V, 0, s, pl), df[s]);
        const int lo = j0 - (S.qw + 31 + S.shift), hi = j0 + TK - 1 - (S.qw + S.shift);
        const bool near = BIAS && !(lo >= A.far_hi || hi <= A.far_lo);
        if (near) {
            floatx16 bias;
            table.block<true>(bias, A, j0, i, g);
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = fmaf(x[r], A.scale2, bias[r] - lse2);
        } else {
            const float bias = (!BIAS ? 0.0f : table.beyond(hi <= A.far_lo)) - lse2;
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = fmaf(x[r], A.scale2, bias);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) y[r] = exp2_fast(x[r]) * (y[r] - delta);
        if (j0 + TK > S.nwave_lo) {
#pragma unroll
            for (int r = 0; r < 16; ++r) y[r] = j0 + block_row(r, g) >= S.nlane ? 0.0f : y[r];
        }
        if constexpr (BIAS) {
            if (near) {
                const int base = j0 - (S.qw + S.shift), off = base + lane - 32;
                const int id = A.near_n ? Ids[off - A.far_lo + kAttnPad] : Bias::bucket_of(A.borders, off);
                near_bias(y, Ss + wave * 32 * kDiagPitch, Dg + wave * 64, base, id, range, near_sum, lane);
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
            for (int d = 0; d < DC / 32; ++d) Ops<T>::mma(dq[d], Kt::col_frag(K, 16 * s, d, pl), ds);
        }
    });
    if constexpr (BIAS) {
#pragma unroll
        for (int w = 1; w < 64; w *= 2) {
            far_lo_sum += __shfl_xor(far_lo_sum, w, 64);
            far_hi_sum += __shfl_xor(far_hi_sum, w, 64);
        }
        float* part = A.part + ((S.bh * A.qtiles + S.qt) * 4 + wave) * A.buckets;
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
    if constexpr (DEEP) {
        join_waves<T, DC>(dq, A.scale, reinterpret_cast<float*>(K0), reinterpret_cast<float*>(V0), wave, lane,
                          i < A.len_q, A.dim, [&]() { return at_row<T>(A.dq, S.b, i, S.h); });
    } else {
        if (i >= A.len_q) return;
        store_rows<T, DC>(at_row<T>(A.dq, S.b, i, S.h), dq, A.scale, A.dim, lane);
    }
}

// For stretches too long for the LDS table (kAttnNear): a launch more and
// scores' bias from global memory.  Used for every stretch instead of the
// table, 77 rows, 4 heads of 32 take 12.4 us instead of 8.8, 8 sequences of
// 512 forward 25.6 instead of 22.0.
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

// Blocks of 32 queries per step of the pass by keys: two where the registers
// hold them beside two waves per SIMD (8 sequences of 512, 16 heads of 64: 28.5
// us, with one 31).
template <typename T, int DC>
constexpr int query_blocks() {
    return sizeof(T) == 2 && DC <= 64 ? 2 : 1;
}

// The grid whose workgroups turn_item() numbers: `run` items of each key and
// value head.  A turn is a whole number of heads, and a multiple of eight
// workgroups, which keeps a workgroup's XCD its number's last three bits.
dim3 turns(const AttnArgs& a, int64_t run) {
    const int64_t heads = (int64_t)a.batch * a.kv_heads;
    int64_t t = std::min<int64_t>(heads / 8, 64);
    while (t > 1 && (heads % t != 0 || heads / t * run % 8 != 0)) --t;
    t = std::max<int64_t>(t, 1);
    return dim3((unsigned)(heads / t * run), (unsigned)t);
}

}  // namespace

int attn_step_queries(bool bf16, int dim) {
    int n = 0;
    by_form(bf16, dim, false, [&](auto* t, auto dc, auto) {
        n = 32 * query_blocks<std::remove_pointer_t<decltype(t)>, decltype(dc)::value>();
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
        const dim3 grid = turns(a, (int64_t)a.group * a.qtiles);
        constexpr int DC = decltype(dc)::value;
        constexpr bool BIAS = decltype(bias)::value;
        if (a.deep) hipLaunchKernelGGL((attn_forward_kernel<T, DC, BIAS, true>), grid, dim3(NT), 0, stream, a);
        else hipLaunchKernelGGL((attn_forward_kernel<T, DC, BIAS, false>), grid, dim3(NT), 0, stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_attn_dq(const AttnArgs& a, bool bf16, hipStream_t stream) {
    by_form(bf16, a.dim, a.buckets != 0, [&](auto* t, auto dc, auto bias) {
        using T = std::remove_pointer_t<decltype(t)>;
        const dim3 grid = turns(a, (int64_t)a.group * a.qtiles);
        constexpr int DC = decltype(dc)::value;
        constexpr bool BIAS = decltype(bias)::value;
        if (a.deep) hipLaunchKernelGGL((attn_dq_kernel<T, DC, BIAS, true>), grid, dim3(NT), 0, stream, a);
        else hipLaunchKernelGGL((attn_dq_kernel<T, DC, BIAS, false>), grid, dim3(NT), 0, stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_attn_dkdv(const AttnArgs& a, bool bf16, hipStream_t stream) {
    by_form(bf16, a.dim, a.buckets != 0, [&](auto* t, auto dc, auto bias) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int DC = decltype(dc)::value;
        const int64_t sums = (int64_t)a.buckets * a.heads;
        dim3 grid = turns(a, (int64_t)a.parts * a.ktiles);
        // (more sums than a grid's second index counts beside short turns: one turn)
        if (grid.x != 0 && ceil_div(sums, grid.x) + grid.y > 65535) grid = dim3(grid.x * grid.y);
        if (grid.x == 0) grid = dim3((unsigned)sums);
        else grid.y += (unsigned)ceil_div(sums, grid.x);
        if (grid.x != 0)
            hipLaunchKernelGGL((attn_dkdv_kernel<T, DC, query_blocks<T, DC>(), decltype(bias)::value>), grid, dim3(NT), 0,
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
