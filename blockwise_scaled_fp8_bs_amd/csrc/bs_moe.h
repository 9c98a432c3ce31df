// Internal interface of the kernels around the experts' products: routing,
// the sort of the routed slots by expert, the gather fused with the
// quantizer, and the combine (bs_moe.hip).  Arguments arrive validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bs {

constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopK = 32;
constexpr int64_t kMaxAlign = 65536;  // rows that a group is padded to a multiple of

struct RouteArgs {
    const void* logits;  // [T, ld] fp32 or bf16
    bool bf16;
    int64_t T, E, ld;
    const float* bias;  // [E] or NULL
    bool sigmoid;
    int32_t k, n_group, topk_group, group_best;
    bool renorm;
    float scale;
    int32_t* idx;  // [T, k]
    float* w;      // [T, k]
    bool vec, vec_bias;  // 16-byte loads of the logits' rows, of the bias
    int32_t lds_token;   // floats of LDS of a token (set by the launcher)
};

struct RouteBwdArgs {
    const void* logits;
    bool bf16;
    int64_t T, E, ld;
    bool sigmoid;
    int32_t k;
    bool renorm;
    float scale;
    const int32_t* idx;
    const float *w, *dw;
    void* dlogits;  // [T, ld_d], the type of logits
    int64_t ld_d;
    bool vec, vec_d;
};

struct PlanArgs {
    const int32_t* idx;  // [T * k]
    int64_t n;           // T * k
    int32_t E, align;
    int64_t M;
    int32_t *group_end, *counts, *slot_row, *row_slot;
    int32_t* hist;  // workspace [blocks][E] (NULL when blocks == 1)
    int32_t blocks, chunks;  // each block sorts 512 * chunks slots
};

struct GatherArgs {
    const uint16_t* x;
    int64_t T, D, ld_x;
    int32_t k;
    uint32_t k_mul, k_shift;  // slot / k = k_mul ? umulhi(slot, k_mul) >> k_shift : slot
    const int32_t* row_slot;
    int64_t M;
    const float* w;  // [T * k] or NULL
    uint16_t* y;
    int64_t ld_y;
    uint8_t* q_row;
    int64_t ld_qr;
    float* s_row;
    int64_t ld_sr;
    uint8_t* q_col;
    int64_t ld_qc;
    float* s_col;
    int64_t ld_sc;
};

struct CombineArgs {
    const uint16_t* y;
    int64_t M, D, ld_y;
    const int32_t* slot_row;  // [T, k]
    const float* w;           // [T, k] or NULL (all ones)
    int64_t T;
    int32_t k;
    const uint16_t* residual;
    int64_t ld_res;
    uint16_t* out;
    int64_t ld_out;
};

struct CombineDwArgs {
    const uint16_t* dout;
    int64_t ld_dout;
    const uint16_t* y;
    int64_t M, D, ld_y;
    const int32_t* slot_row;
    int64_t T;
    int32_t k;
    float* dw;
};

// Slots that one block of the plan sorts, and the blocks for n slots.
void plan_blocks(int64_t n, int32_t* blocks, int32_t* chunks);

hipError_t launch_route(const RouteArgs& a, hipStream_t stream);
hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t stream);
hipError_t launch_plan(const PlanArgs& a, hipStream_t stream);
hipError_t launch_gather(const GatherArgs& a, hipStream_t stream);
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream);
hipError_t launch_combine_dw(const CombineDwArgs& a, hipStream_t stream);

}  // namespace bs
