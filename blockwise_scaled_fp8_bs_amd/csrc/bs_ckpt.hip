// The gated activation that keeps its inputs in 8 bits, for gfx950: the
// forward pass quantizes a and b along their rows from the same read that
// makes h = silu(a) b and its codes; the backward pass reads those codes and
// scales instead of the bf16 pair, half the bytes, and what a training step
// holds between the passes is a little over half.
//
// Both work on 128x128 tiles as the quantizers do, one tile per workgroup,
// and keep their arithmetic: fp32, with the float64 formula where the fp32
// result lies near a bf16 rounding tie, so h, da and db are the float64
// values of their formulas rounded once.
#include "bs_norm.h"
#include "bs_tile.h"

namespace bs {

namespace {

template <bool ROW, bool COL>
__global__ __launch_bounds__(kThreads) void swiglu_ckpt_kernel(SwigluCkptArgs a) {
    __shared__ float s_colmax[4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[COL ? kTile * kTile : 16];
    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int64_t col_tiles = a.C / kTile;
    const int64_t r0 = (blockIdx.x / col_tiles) * kTile, c0 = (blockIdx.x % col_tiles) * kTile;
    const int64_t rows = (a.R - r0) < kTile ? (a.R - r0) : kTile;
    Raw ra, rb, ph;
    load_raw(a.a, a.ld_a, r0, c0, a.R, (8 * tr) * (int)(a.ld_a * 2) + 16 * tc, ra);
    load_raw(a.b, a.ld_b, r0, c0, a.R, (8 * tr) * (int)(a.ld_b * 2) + 16 * tc, rb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float fa[8], fb[8], g[8];
        unpack8(ra.v[i], fa);
        unpack8(rb.v[i], fb);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = swiglu_fast(fa[j], fb[j]);
        ph.v[i] = make_uint4(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[4], g[5]),
                             pack_bf16(g[6], g[7]));
    }
    TileRegs tl;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int64_t co = (half ? a.C : 0) + c0;
        unpack_tile(half ? rb : ra, tl);
        quant_tile_rows(tl, rows, a.ck + r0 * a.ld_ck + co, a.ld_ck, a.s_ck + (co / kTile) * a.ld_sck + r0, tr, tc);
    }
    fixup_block(ph, [&](int e) {
        const int64_t r = r0 + 8 * tr + (e >> 3), c = c0 + 8 * tc + (e & 7);
        if (r >= a.R) return;
        raw_set(ph, e, swiglu_bf16_f64(__uint_as_float((uint32_t)a.a[r * a.ld_a + c] << 16),
                                       __uint_as_float((uint32_t)a.b[r * a.ld_b + c] << 16)));
    });
    unpack_tile(ph, tl);
    if (ROW)
        quant_tile_rows(tl, rows, a.q_row + r0 * a.ld_qr + c0, a.ld_qr, a.s_row + (c0 / kTile) * a.ld_sr + r0, tr, tc);
    if (COL)
        quant_tile_cols(tl, a.q_col + c0 * a.ld_qc + r0, a.ld_qc, a.s_col + (r0 / kTile) * a.ld_sc + c0, s_colmax,
                        s_tr, tr, tc, t >> 6);
}

// Two e4m3 codes of a word (its low or high half) -> floats.
__device__ __forceinline__ void decode8(u32x2 w, float s, float* f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
        f[4 * h] = lo[0] * s;
        f[4 * h + 1] = lo[1] * s;
        f[4 * h + 2] = hi[0] * s;
        f[4 * h + 3] = hi[1] * s;
    }
}

__device__ __forceinline__ float decode1(uint8_t c, float s) {
    return __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false)[0] * s;
}

// A checkpointed tile: codes of rows 8 tr .. +7, columns 8 tc .. +7, and those rows' scales.
struct RawCk {
    u32x2 q[8];
    float s[8];
};

__device__ __forceinline__ void load_ck(const uint8_t* ck, int64_t ld, const float* s, int64_t rows, int tr, int tc,
                                        RawCk& o) {
    const __amdgpu_buffer_rsrc_t rq = rsrc(ck, rows * ld), rs = rsrc(s, rows * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o.q[i] = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_raw_buffer_load_b64(rq, (8 * tr) * (int)ld + 8 * tc, i * (int)ld, 0));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o.s[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, (8 * tr + i) * 4, 0, 0));
}

template <bool ROW, bool COL>
__global__ __launch_bounds__(kThreads) void swiglu_bwd_ckpt_kernel(SwigluBwdCkptArgs a) {
    __shared__ float s_colmax[2][4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[COL ? 2 : 1][COL ? kTile * kTile : 16];
    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int64_t col_tiles = a.C / kTile;
    const int64_t r0 = (blockIdx.x / col_tiles) * kTile, c0 = (blockIdx.x % col_tiles) * kTile;
    const int64_t rows = (a.R - r0) < kTile ? (a.R - r0) : kTile;
    RawCk ka, kb;
    Raw rd;
    const float* const sa = a.s_ck + (c0 / kTile) * a.ld_sck + r0;
    const float* const sb = a.s_ck + ((a.C + c0) / kTile) * a.ld_sck + r0;
    load_ck(a.ck + r0 * a.ld_ck + c0, a.ld_ck, sa, rows, tr, tc, ka);
    load_ck(a.ck + r0 * a.ld_ck + a.C + c0, a.ld_ck, sb, rows, tr, tc, kb);
    load_raw(a.dh, a.ld_dh, r0, c0, a.R, (8 * tr) * (int)(a.ld_dh * 2) + 16 * tc, rd);
    Raw pda, pdb;  // da and db packed as bf16 (da marked where undecided)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float fa[8], fb[8], fd[8], ga[8], gb[8];
        decode8(ka.q[i], ka.s[i], fa);
        decode8(kb.q[i], kb.s[i], fb);
        unpack8(rd.v[i], fd);
#pragma unroll
        for (int j = 0; j < 8; ++j) swiglu_grad_fast(fa[j], fb[j], fd[j], ga[j], gb[j]);
        pda.v[i] = make_uint4(pack_bf16(ga[0], ga[1]), pack_bf16(ga[2], ga[3]), pack_bf16(ga[4], ga[5]),
                              pack_bf16(ga[6], ga[7]));
        pdb.v[i] = make_uint4(pack_bf16(gb[0], gb[1]), pack_bf16(gb[2], gb[3]), pack_bf16(gb[4], gb[5]),
                              pack_bf16(gb[6], gb[7]));
    }
    fixup_block(pda, [&](int e) {
        const int rl = 8 * tr + (e >> 3);
        const int64_t r = r0 + rl, c = c0 + 8 * tc + (e & 7);
        if (r >= a.R) return;
        const float2 g = swiglu_grad_bf16_f64(decode1(a.ck[r * a.ld_ck + c], sa[rl]),
                                              decode1(a.ck[r * a.ld_ck + a.C + c], sb[rl]),
                                              __uint_as_float((uint32_t)a.dh[r * a.ld_dh + c] << 16));
        raw_set(pda, e, g.x);
        raw_set(pdb, e, g.y);
    });
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int64_t co = (half ? a.C : 0) + c0;
        TileRegs tl;
        unpack_tile(half ? pdb : pda, tl);
        if (ROW)
            quant_tile_rows(tl, rows, a.q_row + r0 * a.ld_qr + co, a.ld_qr, a.s_row + (co / kTile) * a.ld_sr + r0, tr,
                            tc);
        if (COL)
            quant_tile_cols(tl, a.q_col + co * a.ld_qc + r0, a.ld_qc, a.s_col + (r0 / kTile) * a.ld_sc + co,
                            s_colmax[half], s_tr[half], tr, tc, t >> 6);
    }
}

}  // namespace

hipError_t launch_swiglu_ckpt(const SwigluCkptArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((a.R + kTile - 1) / kTile) * (a.C / kTile))), block(kThreads);
    if (a.q_row && a.q_col) hipLaunchKernelGGL((swiglu_ckpt_kernel<true, true>), grid, block, 0, stream, a);
    else if (a.q_row) hipLaunchKernelGGL((swiglu_ckpt_kernel<true, false>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((swiglu_ckpt_kernel<false, true>), grid, block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_swiglu_bwd_ckpt(const SwigluBwdCkptArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((a.R + kTile - 1) / kTile) * (a.C / kTile))), block(kThreads);
    if (a.q_row && a.q_col) hipLaunchKernelGGL((swiglu_bwd_ckpt_kernel<true, true>), grid, block, 0, stream, a);
    else if (a.q_row) hipLaunchKernelGGL((swiglu_bwd_ckpt_kernel<true, false>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((swiglu_bwd_ckpt_kernel<false, true>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace bs
