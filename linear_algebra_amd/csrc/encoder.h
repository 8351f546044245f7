// Internal declarations of the operators around an encoder layer's products:
// layer norm, the gated feed-forward block, the norm of many gradients.
// Shared by the host side (encoder_api.hip) and the kernels.
#pragma once

#include "internal.h"

namespace kfac {

// ------------------------------------------------------------- layer norm --
struct NormArgs {
    const void* x;
    const void* dy;
    void* y;                // forward: the output; backward: dx, or nullptr
    int64_t x_stride, dy_stride, y_stride;   // elements from row to row
    float* mean;            // [rows]; forward: or nullptr, rstd likewise
    float* rstd;
    const void* weight;     // [d] or nullptr
    const void* bias;
    void* dweight;          // [d] or nullptr
    void* dbias;
    float* part;            // workspace [parts][2][pitch]: each workgroup's sums of dy xh and dy, or nullptr
    int64_t rows;
    int32_t d, pitch, parts;
    float eps;
};
constexpr int kNormMaxParts = 512;   // workgroups of a backward pass
inline int32_t norm_pitch(int64_t d) { return (int32_t)((d + 3) & ~(int64_t)3); }
// workgroups of the backward pass
int64_t norm_parts(int64_t rows, int64_t d);
hipError_t launch_norm_forward(const NormArgs& a, bool bf16, bool weight_bf16, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs& a, bool bf16, bool weight_bf16, hipStream_t stream);
// dweight and dbias from the workgroups' sums
hipError_t launch_norm_sums(const NormArgs& a, bool weight_bf16, hipStream_t stream);

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
    ClipTensor t[kClipGroup];
};
static_assert(sizeof(ClipTable) <= 4096, "arguments of a launch");
hipError_t launch_clip_squares(const ClipTable& t, int blocks, hipStream_t stream);
hipError_t launch_clip_norm(const ClipTable& t, hipStream_t stream);
hipError_t launch_clip_scale(const ClipTable& t, int blocks, hipStream_t stream);

}  // namespace kfac
