// Internal declarations of the operators that train an encoder layer:
// attention with a bucketed relative position bias, and layer inputs kept in
// 8 bits.  Shared by the host side (training_api.hip) and the kernels.
#pragma once

#include "internal.h"

namespace kfac {

// -------------------------------------------------------------- attention --
constexpr int kAttnThreads = 256;       // 4 waves
constexpr int kAttnRows = 128;          // queries (dQ, forward) or keys (dK, dV) per workgroup, 32 per wave
constexpr int kAttnMaxDim = 128;
constexpr int kAttnMaxBuckets = 128;    // of both sides together: two per lane in the bias gradient

// One tensor [batch, length, heads, dim], dim contiguous, strides in elements.
struct AttnTensor {
    void* p;
    int64_t sb, sl, sh;
};

// Distances at which the buckets of one side begin (the first at 0); INT32_MAX
// from n on.
struct AttnBorders {
    int32_t n, two_sided;
    int32_t at[kAttnMaxBuckets];
};

// Offsets key - query position within kAttnPad of the stretch where the bucket
// changes, in an LDS table, where they are at most kAttnNear.
constexpr int kAttnPad = 96;
constexpr int kAttnNear = 2048;

struct AttnArgs {
    AttnTensor q, k, v, out, dout, dq, dk, dv;
    float* lse;             // [batch][heads][len_q]
    const int32_t* lens;    // visible keys per sequence, or nullptr
    const float* bias;      // [buckets][heads]
    float* dbias;
    float* rel;             // workspace [heads][rel_ld]: bias log2(e) by offset key - query, or nullptr
    float* stats;           // workspace [batch * heads][lq_pad / 32][2][32]: -lse / scale and -delta = -dout . out
                            // of each query (-inf as the first for rows that see nothing or lie past the last)
    float* part;            // workspace [batch * heads][q tiles * 4][buckets]: bias gradient of each wave
    float* kv_part;         // workspace [2][parts][batch * kv_heads][len_k][dim]: shares of dk and dv (parts > 1)
    int64_t rel_ld;
    int32_t batch, len_q, len_k, heads, kv_heads, group, dim;
    int32_t lq_pad;         // len_q rounded up to kAttnRows
    int32_t qtiles, ktiles;
    int32_t deep;           // the passes by queries take 32 queries per workgroup, its waves sharing out the keys
    int32_t causal;
    int32_t buckets;        // 0: no bias
    int32_t far_lo, far_hi; // offsets <= far_lo share one bucket, offsets >= far_hi share one
    int32_t far_lo_bucket, far_hi_bucket;
    int32_t near_n;         // entries of the LDS table, from offset far_lo - kAttnPad on (0: rel instead)
    int32_t parts;          // shares of each key tile: query heads of the group times query chunks
    int32_t qchunk;         // steps of queries per chunk
    float scale, scale2;    // scale2 = scale log2(e)
    AttnBorders borders;
};

hipError_t launch_attn_bias(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_forward(const AttnArgs& a, bool bf16, hipStream_t stream);
// dQ and each wave's share of the bias gradient; leaves stats for launch_attn_dkdv.
hipError_t launch_attn_dq(const AttnArgs& a, bool bf16, hipStream_t stream);
// dK, dV (or their shares) and, in workgroups of its own, the bias gradient's sum.
hipError_t launch_attn_dkdv(const AttnArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_attn_kv_sum(const AttnArgs& a, bool bf16, hipStream_t stream);
// queries per step of launch_attn_dkdv
int attn_step_queries(bool bf16, int dim);

// ------------------------------------------------------------- checkpoints --
// A kept input: e4m3 codes [blocks][da][32] (32 consecutive rows of a column)
// and one scale byte per block and column, [blocks][da], its exponent + 127.
constexpr int kKeepBlock = 32;
constexpr int kKeepMinExp = -117;   // the smallest code times 2^-117 is still a normal bfloat16
constexpr int kKeepGroup = 8;       // layers per launch, passed by value

struct KeepLayer {
    void* x;              // [rows][cols]
    uint8_t* codes;
    uint8_t* scales;
    int64_t rows;
    int64_t block_begin;  // first workgroup of this layer
    int32_t cols;         // columns of x
    int32_t da;           // columns of the checkpoint
    int32_t groups;       // workgroups per block of 32 rows (store) or 16 rows (load)
};
struct KeepLaunch {
    int32_t n;
    KeepLayer layer[kKeepGroup];
};
constexpr int kKeepThreads = 256;
hipError_t launch_keep_store(const KeepLaunch& l, int64_t blocks, bool bf16, hipStream_t stream);
hipError_t launch_keep_load(const KeepLaunch& l, int64_t blocks, bool bf16, hipStream_t stream);

// Products with kept inputs on 128 x 128 tiles.
constexpr int kKeepTile = 128;
struct KeepProb {
    const void* g;        // [rows][m] output gradients (gradient products)
    const uint8_t* codes;
    const uint8_t* scales;
    float* out;           // factor [da][da], or gradient [m][da]
    float* part;          // partial tiles [ksplit][ntiles - whole][128][128]
    int64_t rows;
    int64_t item_begin, red_begin;
    int32_t m;            // rows of the output (da for a factor)
    int32_t da;
    int32_t blocks;       // blocks of 32 rows
    int32_t tiles_m, tiles_n, ntiles;
    int32_t whole;            // tiles [0, whole) in one item each, the others in
    int32_t ksplit, kchunk;   // ksplit chunks of kchunk blocks (even)
    float alpha;
};
struct KeepProbs {
    int32_t n;
    int32_t cut;              // items [0, cut) are whole tiles
    int32_t first_step;
    float eps;
    KeepProb p[kKeepGroup];
};
hipError_t launch_keep_factor(const KeepProbs& l, int64_t items, hipStream_t stream);
// words: the rows of every g start on 4-byte boundaries
hipError_t launch_keep_grad(const KeepProbs& l, int64_t items, bool bf16, bool words, hipStream_t stream);
hipError_t launch_keep_reduce(const KeepProbs& l, int64_t tiles, bool factor, hipStream_t stream);

}  // namespace kfac
