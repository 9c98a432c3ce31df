// Internal interface of the residual norms (bs_norm.hip) and of the gated
// activation with an 8-bit checkpoint (bs_ckpt.hip).  Arguments arrive
// validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bs {

constexpr int64_t kMaxNormDim = 16384;

struct ResidNormArgs {
    const uint16_t *x, *u;  // [R, D]; u may be NULL
    int64_t R, D, ld_x, ld_u;
    const void *w_post, *gate, *w_pre;  // [D], [R / rows_per_gate, D], [D]; each may be NULL
    bool w_bf16;
    int64_t ld_gate, rows_per_gate;
    float alpha, eps;
    uint16_t* r;  // [R, D], written when u is given
    int64_t ld_r;
    float *rstd_u, *rstd_r;  // [R], each may be NULL
    uint16_t* h;             // [R, D] or NULL
    int64_t ld_h;
    uint8_t* q_row;
    int64_t ld_qr;
    float* s_row;
    int64_t ld_sr;
    uint8_t* q_col;
    int64_t ld_qc;
    float* s_col;
    int64_t ld_sc;
};

struct ResidNormBwdArgs {
    const uint16_t *r, *u, *dh, *dr;  // u, dr may be NULL; dh NULL without w_pre
    int64_t R, D, ld_r, ld_u, ld_dh, ld_dr;
    const void *w_post, *gate, *w_pre;
    bool w_bf16;
    int64_t ld_gate, rows_per_gate;  // rows_per_gate = R without a gate
    float alpha;
    const float *rstd_u, *rstd_r;
    uint16_t *dx, *du;
    int64_t ld_dx, ld_du;
    float *dw_pre, *dw_post, *dgate;  // [D], [D], [R / rows_per_gate, D]
    float* ws;
};

// How the backward pass splits the rows over workgroups, and the floats of
// workspace that its partial column sums take.
struct NormBwdSplit {
    int64_t blocks;          // workgroups
    int64_t segs;            // gate segments
    int64_t segs_per_block;  // whole segments of a workgroup (chunks == 1), or 1
    int64_t chunks;          // workgroups per segment
    int64_t rows;            // rows of a chunk
};
NormBwdSplit norm_bwd_split(int64_t R, int64_t D, int64_t rows_per_gate);

struct SwigluCkptArgs {
    const uint16_t *a, *b;
    int64_t R, C, ld_a, ld_b;
    uint8_t* ck;  // [R, 2C]
    int64_t ld_ck;
    float* s_ck;  // [2C / 128][ld_sck >= R]
    int64_t ld_sck;
    uint8_t* q_row;
    int64_t ld_qr;
    float* s_row;
    int64_t ld_sr;
    uint8_t* q_col;
    int64_t ld_qc;
    float* s_col;
    int64_t ld_sc;
};

struct SwigluBwdCkptArgs {
    const uint8_t* ck;
    int64_t R, C, ld_ck;
    const float* s_ck;
    int64_t ld_sck;
    const uint16_t* dh;
    int64_t ld_dh;
    uint8_t* q_row;  // [R, 2C]
    int64_t ld_qr;
    float* s_row;
    int64_t ld_sr;
    uint8_t* q_col;  // [2C, R]
    int64_t ld_qc;
    float* s_col;
    int64_t ld_sc;
};

hipError_t launch_resid_norm(const ResidNormArgs& a, hipStream_t stream);
hipError_t launch_resid_norm_bwd(const ResidNormBwdArgs& a, hipStream_t stream);
hipError_t launch_swiglu_ckpt(const SwigluCkptArgs& a, hipStream_t stream);
hipError_t launch_swiglu_bwd_ckpt(const SwigluBwdCkptArgs& a, hipStream_t stream);

}  // namespace bs
