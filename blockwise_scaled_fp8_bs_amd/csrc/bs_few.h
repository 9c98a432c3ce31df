// Internal interface of the kernels that serve few tokens from quantized
// weights (bs_few.hip) and of the MXFP4 quantizer of those weights
// (bs_mx4.hip).  Arguments arrive validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bs {

constexpr int64_t kFewChunk = 64;               // tokens that a workgroup takes at a time
constexpr int kCus = 256;
constexpr int64_t kTwoParts = 8;                // tokens up to which bs_moe_few can keep h in two parts
constexpr int kMaxSplits = 16;                  // workgroups that share columns of bs_moe_few's output
constexpr int64_t kMaxFewDim = (int64_t)1 << 18;  // widths of bs_moe_few: a chunk's slots times them in 32-bit offsets

typedef float few_f32x4 __attribute__((ext_vector_type(4)));

enum FewKind { kFewE4m3 = 0, kFewMx8 = 1, kFewMx4 = 2 };

struct Mx4QuantArgs {
    const uint16_t* x;
    int64_t R, C, ld_x;
    uint8_t* q;  // [R, C / 2]
    int64_t ld_q;
    uint8_t* s;  // [C / 32][ld_s >= R]
    int64_t ld_s;
    uint16_t* y;  // [R, C] or NULL
    int64_t ld_y;
    int64_t col_tiles;
};

// Quantized weights [N, K] (of every expert): strides in elements of their type.
struct FewWeight {
    const uint8_t* q;
    int64_t stride_q, ld_q;  // bytes
    const void* s;
    int64_t stride_s, ld_s;
};

struct FewMmArgs {
    int64_t T, N, K;
    const uint16_t* x;
    int64_t ld_x;
    FewWeight w;
    const uint16_t* residual;  // [T, N] or NULL
    int64_t ld_res;
    void* out;
    int64_t ld_out;
    bool f32, vec;  // type of out; four columns at a time
    int64_t tiles;  // set by the launcher
};

struct MoeFewArgs {
    int64_t T, D, H;
    int32_t E, k;
    const uint16_t* x;
    int64_t ld_x;
    const int32_t* idx;  // [T, k], or NULL: every token takes expert 0
    const float* w;      // [T, k], or NULL: ones
    FewWeight w12, wo;
    const uint16_t* residual;  // [T, D] or NULL
    int64_t ld_res;
    uint16_t* out;
    int64_t ld_out;
    bool vec;
    uint16_t* h;    // workspace [T * k, parts, H] bf16
    int32_t parts;  // that h is kept in
    // set by the launcher
    int64_t tiles;
    int32_t items;      // work items of a chunk at most
    int32_t splits;     // workgroups that share columns of the output
    few_f32x4* part;    // workspace: their sums [splits][T, D]
};

hipError_t launch_mx4_quant(const Mx4QuantArgs& a, hipStream_t stream);
// What a call runs (bs_diag_few_mm_plan and bs_diag_moe_few_plan).
struct FewMmPlan {
    int64_t rows, tiles;          // rows of x and tiles of 16 columns of a workgroup
    int64_t workgroups, threads;  // along the columns; of a workgroup
};
struct MoeFewPlan {
    int64_t tokens, items;  // tokens of an item, items of a chunk, at most
    int64_t up_tiles;       // tiles of h that a wave streams at a time, 0: the waves of a workgroup share one
    int64_t up_waves;       // waves that whole tiles are spread over
    int64_t out_tiles, splits;  // tiles of the output at a time, workgroups that share them
};

// With `plan`: nothing is launched, it says what would be.
hipError_t launch_few_mm(const FewMmArgs& a, FewKind kind, hipStream_t stream, FewMmPlan* plan = nullptr);
hipError_t launch_moe_few(const MoeFewArgs& a, FewKind kind, hipStream_t stream, MoeFewPlan* plan = nullptr);

// Workspace of the workgroups that share columns of the output (0: none can).
int64_t moe_few_shares_bytes(int64_t T, int64_t D, int64_t H, int64_t E, int64_t k);

}  // namespace bs
