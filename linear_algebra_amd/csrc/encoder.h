// Internal declarations of the operators around an encoder layer's products:
// layer norm, the gated feed-forward block, the norm of many gradients.
// Shared by the host side (encoder_api.hip) and the kernels.
#pragma once

#include "internal.h"

namespace kfac {

constexpr int64_t kLastCache = 256 << 20;   // bytes of the chip's last cache

// ------------------------------------------------------------- layer norm --
// Sums of many workgroups over rows, to be added: two vectors of d columns.
struct PartSums {
    const float* part;      // [parts][2][pitch]
    void* dweight;          // [d] or nullptr: the sums of the first
    void* dbias;            // of the second
    int32_t d, pitch, parts;
};
constexpr int kSumColumns = 32;   // per workgroup
inline int sums_blocks(int32_t pitch) { return 2 * ((pitch + kSumColumns - 1) / kSumColumns); }

struct NormArgs {
    const void* x;
    const void* dy;
    void* y;                // forward: the output; backward: dx, or nullptr
    int64_t x_stride, dy_stride, y_stride;   // elements from row to row
    float* mean;            // [rows]; forward: or nullptr, rstd likewise
    float* rstd;
    const void* weight;     // [d] or nullptr
    const void* bias;
    float* part;            // workspace [parts][2][pitch]: each workgroup's sums of dy xh and dy, or nullptr
    int64_t rows;
    int32_t d, pitch, parts;
    float eps;
};
inline int32_t norm_pitch(int64_t d) { return (int32_t)((d + 3) & ~(int64_t)3); }
// workgroups of the backward pass
int64_t norm_parts(int64_t rows, int64_t d, bool bf16);
hipError_t launch_norm_forward(const NormArgs& a, bool bf16, bool weight_bf16, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs& a, bool bf16, bool weight_bf16, hipStream_t stream);
// dweight and dbias from the workgroups' sums
hipError_t launch_norm_sums(const PartSums& a, bool weight_bf16, hipStream_t stream);

// --------------------------------------------------------- gradient norm --
// Gradients are cut into chunks of kClipChunk elements; a launch serves the
// tensors of one table, which travels by value, and its workgroups go through
// the table's chunks in turns.
constexpr int kClipChunk = 8192;
constexpr int kClipThreads = 256;
constexpr int kClipBlocks = 1024;    // workgroups of all launches of a pass together, apart from one per launch
constexpr int kClipGroup = 160;      // tensors per launch: a table of at most 4 KB


struct ClipTensor {
    const void* g;
    void* out;              // may be g
    uint32_t begin;         // first chunk in the table
    uint32_t last;          // elements of the last chunk, and kClipBf16
};
constexpr uint32_t kClipBf16 = 0x80000000u;
struct ClipTable {
    double* part;           // workspace: a sum of squares for each workgroup of every launch
    float* norm;
    int32_t n;              // tensors
    int32_t first_part;     // where this launch's sums begin
    int32_t parts;          // sums of all launches
    uint32_t chunks;
    float max_norm;
    int32_t writes_norm;
    int32_t once;           // the scaling reads and writes past the caches
    ClipTensor t[kClipGroup];
};
static_assert(sizeof(ClipTable) <= 4096, "arguments of a launch");
hipError_t launch_clip_squares(const ClipTable& t, int blocks, hipStream_t stream);
hipError_t launch_clip_norm(const ClipTable& t, hipStream_t stream);
hipError_t launch_clip_scale(const ClipTable& t, int blocks, hipStream_t stream);

// ------------------------------------------------------------------ gated --
constexpr int kActSilu = 0, kActGelu = 1, kActGeluTanh = 2, kActRelu = 3, kActSigmoid = 4;

// A bfloat16 matrix (or the first of three planes): 4-byte aligned rows of an
// even pitch.
struct ProdOperand {
    const uint16_t* p;
    int64_t plane;      // elements from plane to plane
    int64_t bytes;      // of a plane, up to the end of its last row
    int32_t ld;         // elements
    int32_t limit;      // rows that exist (reduction along a row), or columns
    int32_t apart;      // forward: rows from a gate row of W to its up row
};
// out[M][N] = the sum over K, or the gated forward's outputs.
struct ProdArgs {
    ProdOperand a, b;
    int64_t K, kchunk;  // reduction steps, and those of a share
    int32_t M, N;
    int32_t tiles_m, tiles_n, tiles;
    int32_t whole;      // tiles [0, whole) in one item each, the others shared out along K
    int32_t splits;     // shares of each of the others
    int32_t width;      // F
    int32_t act;
    int32_t out_bf16;
    const float* bias;  // [2 F] or nullptr
    void* out;
    void* pre;          // [M][2 F] or nullptr
    float* part;        // workspace [shares][tiles - whole][tile]
};
// The backward pass's products: dx, dW.
struct ProdPair {
    ProdArgs p[2];
};

// The forms of a product.  What one costs was measured on products of 4096 x
// 1024 x 5460 and 25088 x 2304 x 9216: microseconds for 64 reduction steps of
// a tile while every slot of the card holds one, and for what a tile takes
// besides (the last form: on the backward products of 25088 x 2304 -> 4608).
struct ProdForm {
    int m, n;           // rows and columns of a tile (forward: n / 2 columns of each projection)
    int slots;          // workgroups at work at once
    int threads;        // of each
    double step, rest;
};
constexpr int kProdWide = 0;    // 256 x 256 by eight waves: the least LDS traffic for each product
constexpr int kProdPair = 1;    // 128 x 128 by four waves, two workgroups on a compute unit
constexpr int kProdDeep = 2;    // 128 x 128 by four waves, two slabs ahead
constexpr int kProdParts = 3;   // float32, in three parts: 128 x 128 by eight waves
constexpr int kProdMixed = 4;   // float32 dpre against bfloat16: 128 x 128 by four waves
constexpr ProdForm kProdForms[5] = {{256, 256, 256, 512, 1.75, 12.0},
                                    {128, 128, 512, 256, 0.95, 8.0},
                                    {128, 128, 256, 256, 0.65, 6.0},
                                    {128, 128, 256, 512, 2.8, 8.0},
                                    {128, 128, 512, 256, 3.3, 8.0}};
// items: whole tiles and shares
hipError_t launch_gated_forward(const ProdArgs& a, int form, int64_t items, hipStream_t stream);
// the outputs of shared tiles, of which there are some
hipError_t launch_gated_forward_finish(const ProdArgs& a, int form, hipStream_t stream);
hipError_t launch_gated_backward(const ProdPair& a, int form, int64_t items, hipStream_t stream);
// the sums of shared tiles and, where s has an output, of the bias's gradient
hipError_t launch_gated_finish(const ProdPair& a, int form, const PartSums& s, hipStream_t stream);

// The forward product of few rows, from operands of any alignment.
struct RowsArgs {
    const void* x;          // [rows][d]
    const void* weight;     // [2 width][d]
    const float* bias;
    void* h;
    void* pre;
    int64_t rows;
    int32_t d, width, act;
};
constexpr int kRowsWaves = 8;   // of a workgroup, sharing out the reduction
// blocks of 16 rows that a workgroup holds
inline int gated_rows_blocks(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
hipError_t launch_gated_rows(const RowsArgs& a, bool bf16, hipStream_t stream);

struct RepackMatrix {
    const void* src;    // [rows][cols]
    void* dst;          // [rows][pitch], or three such planes
    int64_t rows, plane;
    int32_t cols, pitch;
    uint32_t begin;     // first workgroup
    int32_t bf16;
};
struct RepackTable {
    int32_t n;
    RepackMatrix m[2];
};
hipError_t launch_repack(const RepackTable& t, int64_t blocks, hipStream_t stream);

struct GatedGradArgs {
    const void* dh;     // [rows][width]
    const void* pre;    // [rows][2 width]
    void* dpre;
    float* part;        // workspace [parts][2][pitch] or nullptr
    uint16_t* planes;   // float32 dpre in three parts [3][rows][plane_pitch], or nullptr
    int64_t plane;
    int64_t rows, chunk;
    int32_t width, pitch, act, plane_pitch;
};
hipError_t launch_gated_grad(const GatedGradArgs& a, int parts, bool bf16, bool dpre_bf16, hipStream_t stream);

}  // namespace kfac
