// Blockwise e4m3 quantizer kernels for gfx950.
//
// Every kernel works on 128x128 tiles of a bf16 matrix with 256 threads
// (4 wave64s).  Thread t owns an 8x8 sub-block: rows 8*(t/16) .. +7 and
// columns 8*(t%16) .. +7 of the tile, loaded as eight 16-byte row chunks, so
// a wave reads four full 256-byte row segments per load instruction.
//
//  * 1x128 row blocks: the 16 threads sharing a row group sit in one DPP row
//    of their wave; the block amax is a 4-step DPP max.
//  * 1x128 column blocks (128 consecutive rows of a column): per-thread max
//    over its 8 rows, shuffle over the 4 row groups of a wave, LDS over the 4
//    waves.  The codes are written transposed through an XOR-swizzled LDS
//    tile so that the global stores are full 128-byte rows of q^T.
//  * 128x128 blocks: one amax per tile (thread -> DPP row -> wave -> LDS).
//
// Workgroups are persistent: each walks the tiles with a grid stride and
// loads the next tile's bf16 data into registers before working on the
// current one, so HBM reads overlap the arithmetic and no partly filled last
// wave of workgroups is left (passes over large operands launch one
// workgroup per tile instead: persistent_blocks).  LDS buffers alternate
// between consecutive tiles, so one barrier per LDS exchange suffices.  Each
// tile reads HBM once and writes each requested output once.
#include "bs_kernels.h"
#include "bs_device.h"
#include "bs_mx.h"
#include "bs_tile.h"

namespace bs {

namespace {

// 1x128 quantizer (rows and/or transposed columns).  SWIGLU quantizes
// h = bf16(silu(x) * y) instead of x, from one read of x and y, and writes
// h too when a.h is set.  ONE: the form for a grid of one workgroup per tile
// (the loop then runs once): each tile's inputs are loaded where they are
// used, with no registers held for the next tile's, so that more waves fit
// on a SIMD.
template <bool ROW, bool COL, bool SWIGLU, bool ONE>
__global__ __launch_bounds__(kThreads) void quant_1x128_kernel(Quant1x128Args a) {
    // ONE: a single LDS set (18 KiB instead of 36), a barrier between tiles
    // in the rare case that the grid is smaller than the tile count
    constexpr int kSets = ONE ? 1 : 2;
    __shared__ float s_colmax[kSets][4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[COL ? kSets : 1][COL ? kTile * kTile : 16];

    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int wave = t >> 6;
    const int64_t ntiles = ((a.R + kTile - 1) / kTile) * a.col_tiles;

    int64_t tile = blockIdx.x;
    if (tile >= ntiles) return;
    const int voff_x = (8 * tr) * (int)(a.ld_x * 2) + 16 * tc;
    const int voff_y = SWIGLU ? (8 * tr) * (int)(a.ld_y * 2) + 16 * tc : 0;
    Raw raw, raw_y;
    if (!ONE) {
        load_raw(a.x, a.ld_x, (tile / a.col_tiles) * kTile, (tile % a.col_tiles) * kTile, a.R, voff_x, raw);
        if (SWIGLU)
            load_raw(a.y, a.ld_y, (tile / a.col_tiles) * kTile, (tile % a.col_tiles) * kTile, a.R, voff_y, raw_y);
    }

    for (int parity = 0; tile < ntiles; tile += gridDim.x, parity ^= 1) {
        const int64_t r0 = (tile / a.col_tiles) * kTile, c0 = (tile % a.col_tiles) * kTile;
        const int64_t rows = (a.R - r0) < kTile ? (a.R - r0) : kTile;
        if (ONE) {
            load_raw(a.x, a.ld_x, r0, c0, a.R, voff_x, raw);
            if (SWIGLU) load_raw(a.y, a.ld_y, r0, c0, a.R, voff_y, raw_y);
        }
        TileRegs tl;
        Raw ph;  // gated form: h packed as bf16, +inf where the fp32 path left it undecided
        if (SWIGLU) {
            // row by row from the packed inputs, so that no float tile is live
            // while the next tile's inputs are loaded
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float fa[8], fb[8], g[8];
                unpack8(raw.v[i], fa);
                unpack8(raw_y.v[i], fb);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = swiglu_fast(fa[j], fb[j]);
                ph.v[i] = make_uint4(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[4], g[5]),
                                     pack_bf16(g[6], g[7]));
            }
        } else {
            unpack_tile(raw, tl);
        }
        const int64_t next = tile + gridDim.x;
        if (!ONE && next < ntiles) {
            load_raw(a.x, a.ld_x, (next / a.col_tiles) * kTile, (next % a.col_tiles) * kTile, a.R, voff_x, raw);
            if (SWIGLU)
                load_raw(a.y, a.ld_y, (next / a.col_tiles) * kTile, (next % a.col_tiles) * kTile, a.R, voff_y,
                         raw_y);
        }
        if (SWIGLU) {
            // undecided elements: their inputs are read again (a few per tile)
            // and h is recomputed in float64
            fixup_block(ph, [&](int e) {
                const int64_t r = r0 + 8 * tr + (e >> 3), c = c0 + 8 * tc + (e & 7);
                if (r >= a.R) return;  // rows past the end read as zeros and are never marked
                raw_set(ph, e, swiglu_bf16_f64(__uint_as_float((uint32_t)a.x[r * a.ld_x + c] << 16),
                                                     __uint_as_float((uint32_t)a.y[r * a.ld_y + c] << 16)));
            });
            if (a.h != nullptr) store_raw(ph, a.h + r0 * a.ld_h + c0, a.ld_h, rows, tr, tc);
            unpack_tile(ph, tl);
        }
        if (ROW) quant_tile_rows(tl, rows, a.q_row + r0 * a.ld_qr + c0, a.ld_qr, a.s_row + (c0 / kTile) * a.ld_sr + r0, tr, tc);
        if (COL) {
            quant_tile_cols(tl, a.q_col + c0 * a.ld_qc + r0, a.ld_qc, a.s_col + (r0 / kTile) * a.ld_sc + c0,
                            s_colmax[ONE ? 0 : parity], s_tr[ONE ? 0 : parity], tr, tc, wave);
            if (ONE && tile + gridDim.x < ntiles) __syncthreads();
        }
    }
}

// Backward of the gated activation fused with the 1x128 quantizer: from one
// read of a, b and dh ([R, C] bf16) it forms da and db (each rounded once to
// bf16) and quantizes the [R, 2C] matrix [da | db] along rows and/or its
// transposed columns; [da | db] itself is written when a.dab is set.  Each
// input tile gives two output tiles: da's at columns c0, db's at C + c0.
template <bool ROW, bool COL>
__global__ __launch_bounds__(kThreads) void swiglu_bwd_quant_kernel(SwigluBwdArgs a) {
    __shared__ float s_colmax[2][4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[COL ? 2 : 1][COL ? kTile * kTile : 16];

    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int wave = t >> 6;
    const int64_t ntiles = ((a.R + kTile - 1) / kTile) * a.col_tiles;

    int64_t tile = blockIdx.x;
    if (tile >= ntiles) return;
    const int voff_a = (8 * tr) * (int)(a.ld_a * 2) + 16 * tc;
    const int voff_b = (8 * tr) * (int)(a.ld_b * 2) + 16 * tc;
    const int voff_d = (8 * tr) * (int)(a.ld_dh * 2) + 16 * tc;
    auto load3 = [&](int64_t tl_id, Raw& ra, Raw& rb, Raw& rd) {
        const int64_t r0 = (tl_id / a.col_tiles) * kTile, c0 = (tl_id % a.col_tiles) * kTile;
        load_raw(a.a, a.ld_a, r0, c0, a.R, voff_a, ra);
        load_raw(a.b, a.ld_b, r0, c0, a.R, voff_b, rb);
        load_raw(a.dh, a.ld_dh, r0, c0, a.R, voff_d, rd);
    };
    int parity = 0;
    for (; tile < ntiles; tile += gridDim.x) {
        const int64_t r0 = (tile / a.col_tiles) * kTile, c0 = (tile % a.col_tiles) * kTile;
        const int64_t rows = (a.R - r0) < kTile ? (a.R - r0) : kTile;
        const int64_t C = a.col_tiles * kTile;
        // No prefetch of the next tile: a, b and dh of two tiles would not fit
        // beside the outputs; two workgroups per SIMD hide the latency instead.
        Raw ra, rb, rd;
        load3(tile, ra, rb, rd);
        Raw pda, pdb;  // da and db of the tile, packed bf16 (da marked where undecided)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float fa[8], fb[8], fd[8], ga[8], gb[8];
            unpack8(ra.v[i], fa);
            unpack8(rb.v[i], fb);
            unpack8(rd.v[i], fd);
#pragma unroll
            for (int j = 0; j < 8; ++j) swiglu_grad_fast(fa[j], fb[j], fd[j], ga[j], gb[j]);
            pda.v[i] = make_uint4(pack_bf16(ga[0], ga[1]), pack_bf16(ga[2], ga[3]), pack_bf16(ga[4], ga[5]),
                                  pack_bf16(ga[6], ga[7]));
            pdb.v[i] = make_uint4(pack_bf16(gb[0], gb[1]), pack_bf16(gb[2], gb[3]), pack_bf16(gb[4], gb[5]),
                                  pack_bf16(gb[6], gb[7]));
        }
        // undecided elements: their inputs are read again (a few per tile)
        fixup_block(pda, [&](int e) {
            const int64_t r = r0 + 8 * tr + (e >> 3), c = c0 + 8 * tc + (e & 7);
            if (r >= a.R) return;  // rows past the end read as zeros and are never marked
            const float2 g = swiglu_grad_bf16_f64(__uint_as_float((uint32_t)a.a[r * a.ld_a + c] << 16),
                                                  __uint_as_float((uint32_t)a.b[r * a.ld_b + c] << 16),
                                                  __uint_as_float((uint32_t)a.dh[r * a.ld_dh + c] << 16));
            raw_set(pda, e, g.x);
            raw_set(pdb, e, g.y);
        });
        if (a.dab != nullptr) {
            store_raw(pda, a.dab + r0 * a.ld_dab + c0, a.ld_dab, rows, tr, tc);
            store_raw(pdb, a.dab + r0 * a.ld_dab + C + c0, a.ld_dab, rows, tr, tc);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int64_t co = (half ? C : 0) + c0;  // output column of the tile
            TileRegs tl;
            unpack_tile(half ? pdb : pda, tl);
            if (ROW)
                quant_tile_rows(tl, rows, a.q_row + r0 * a.ld_qr + co, a.ld_qr, a.s_row + (co / kTile) * a.ld_sr + r0,
                                tr, tc);
            if (COL) {
                quant_tile_cols(tl, a.q_col + co * a.ld_qc + r0, a.ld_qc, a.s_col + (r0 / kTile) * a.ld_sc + co,
                                s_colmax[parity], s_tr[parity], tr, tc, wave);
                parity ^= 1;
            }
        }
    }
}

// ---- MXFP8 (OCP Microscaling reading): 32-element blocks, E8M0 scales ----
// E8M0 byte of a block, floor(log2(amax)) - 8 + 127, from amax's exponent
// field; an amax below 2^-119 (scale exponent under -127), a subnormal amax
// or zero gives the smallest scale, byte 0.
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
    const uint32_t ex = (__float_as_uint(amax) >> 23) & 0xFFu;
    return ex > 8u ? ex - 8u : 0u;
}

// Four elements divided by 2^(byte - 127) (exact: a power-of-two scaling),
// saturated at +-448, encoded (round to nearest even, sign kept).
__device__ __forceinline__ uint32_t mx_encode4(float x0, float x1, float x2, float x3, uint32_t byte) {
    const int ne = 127 - (int)byte;
    return encode4(clamp448(__builtin_amdgcn_ldexpf(x0, ne)), clamp448(__builtin_amdgcn_ldexpf(x1, ne)),
                   clamp448(__builtin_amdgcn_ldexpf(x2, ne)), clamp448(__builtin_amdgcn_ldexpf(x3, ne)));
}

// MX quantizer over 128x128 tiles: ROW writes 32-element blocks along each
// row (q_row [R, C], s_row[(c / 32) * ld_sr + r]); COL writes blocks of 32
// consecutive rows of each column, transposed (q_col [C, R],
// s_col[(r / 32) * ld_sc + c]).  A row block spans the 4 threads of a lane
// quad (8 columns each); a column block spans the 4 row groups of one wave.
template <bool ROW, bool COL>
__global__ __launch_bounds__(kThreads) void mx_quant_kernel(MxQuantArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[COL ? 2 : 1][COL ? kTile * kTile : 16];

    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int64_t ntiles = ((a.R + kTile - 1) / kTile) * a.col_tiles;

    int64_t tile = blockIdx.x;
    if (tile >= ntiles) return;
    const int voff_x = (8 * tr) * (int)(a.ld_x * 2) + 16 * tc;
    Raw raw;
    load_raw(a.x, a.ld_x, (tile / a.col_tiles) * kTile, (tile % a.col_tiles) * kTile, a.R, voff_x, raw);

    for (int parity = 0; tile < ntiles; tile += gridDim.x, parity ^= 1) {
        const int64_t r0 = (tile / a.col_tiles) * kTile, c0 = (tile % a.col_tiles) * kTile;
        const int64_t rows = (a.R - r0) < kTile ? (a.R - r0) : kTile;
        TileRegs tl;
        unpack_tile(raw, tl);
        const int64_t next = tile + gridDim.x;
        if (next < ntiles)
            load_raw(a.x, a.ld_x, (next / a.col_tiles) * kTile, (next % a.col_tiles) * kTile, a.R, voff_x, raw);

        if (ROW) {
            const __amdgpu_buffer_rsrc_t rq = rsrc(a.q_row + r0 * a.ld_qr + c0, rows * a.ld_qr);
            const int voff_q = (8 * tr) * (int)a.ld_qr + 8 * tc;
            // scale bytes of the tile's 4 column blocks (the lane quad of columns 8tc.. shares block tc / 4):
            // uniform descriptor over the 4 scale rows, the block in the lane offset, rows checked explicitly
            const __amdgpu_buffer_rsrc_t rs = rsrc(a.s_row + (c0 / 32) * a.ld_sr + r0, 3 * a.ld_sr + rows);
            const int voff_s = (tc / 4) * (int)a.ld_sr;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(tl.f[i][j]));
                uint32_t mb = __float_as_uint(m);
                mb = max(mb, (uint32_t)__builtin_amdgcn_mov_dpp((int)mb, 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
                mb = max(mb, (uint32_t)__builtin_amdgcn_mov_dpp((int)mb, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
                const uint32_t byte = mx_scale_byte(__uint_as_float(mb));
                const uint32_t lo = mx_encode4(tl.f[i][0], tl.f[i][1], tl.f[i][2], tl.f[i][3], byte);
                const uint32_t hi = mx_encode4(tl.f[i][4], tl.f[i][5], tl.f[i][6], tl.f[i][7], byte);
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{lo, hi}, rq, voff_q, i * (int)a.ld_qr, 0);
                // one byte store per row: rows past the end are dropped, nothing beyond is written
                if ((tc & 3) == 0 && 8 * tr + i < rows)
                    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)byte, rs, voff_s + 8 * tr + i, 0, 0);
            }
        }
        if (COL) {
            uint2 codes[8];
            uint32_t bytes[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(tl.f[i][j]));
                m = fmaxf(m, __shfl_xor(m, 16));
                m = fmaxf(m, __shfl_xor(m, 32));
                bytes[j] = mx_scale_byte(m);
                codes[j].x = mx_encode4(tl.f[0][j], tl.f[1][j], tl.f[2][j], tl.f[3][j], bytes[j]);
                codes[j].y = mx_encode4(tl.f[4][j], tl.f[5][j], tl.f[6][j], tl.f[7][j], bytes[j]);
            }
            if ((t & 63) < 16) {  // row group 0 of each wave: the 8 columns' scale bytes of the wave's 32 rows
                const __amdgpu_buffer_rsrc_t rs = rsrc(a.s_col + (r0 / 32 + wave) * a.ld_sc + c0, kTile);
                const uint32_t w0 = bytes[0] | (bytes[1] << 8) | (bytes[2] << 16) | (bytes[3] << 24);
                const uint32_t w1 = bytes[4] | (bytes[5] << 8) | (bytes[6] << 16) | (bytes[7] << 24);
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{w0, w1}, rs, 8 * tc, 0, 0);
            }
            store_transposed(s_tr[parity], codes, tr, tc, a.q_col + c0 * a.ld_qc + r0, a.ld_qc);
        }
    }
}

// 128x128 quantizer.  MODE kQ128Rows writes the codes in place (q, s),
// kQ128Transposed writes each tile transposed (3-D colwise: q, s), kQ128Both
// writes both from one read of x (rows to q, s; transposed to qt, st).
// One 128x128 tile of expert g (tile row rt, column ct) from its values tl:
// the block amax (through wmax, 4 floats of LDS), the scale, and the codes in
// the requested layouts (the transposed ones staged through tr_lds).
template <int MODE>
__device__ __forceinline__ void quant_128_tile(const Quant128Args& a, int64_t g, int64_t rt, int64_t ct,
                                               const TileRegs& tl, float* wmax, uint8_t* tr_lds, int t, int tr,
                                               int tc, int wave) {
    constexpr bool ROWS = MODE != kQ128Transposed;
    constexpr bool TRANSPOSE = MODE != kQ128Rows;
    const int64_t r0 = rt * kTile, c0 = ct * kTile;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(tl.f[i][j]));
    uint32_t mb = row16_max(__float_as_uint(m));
    mb = max(mb, (uint32_t)__shfl_xor((int)mb, 16));
    mb = max(mb, (uint32_t)__shfl_xor((int)mb, 32));
    if ((t & 63) == 0) wmax[wave] = __uint_as_float(mb);
    __syncthreads();
    const float amax = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
    const Scale sc = block_scale(amax);

    if (ROWS) {
        uint8_t* q = a.q + g * a.stride_qg;
        const __amdgpu_buffer_rsrc_t rq = rsrc(q + r0 * a.ld_q + c0, (kTile - 1) * a.ld_q + kTile);
        const int voff_q = (8 * tr) * (int)a.ld_q + 8 * tc;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint2 c8 = quant8(tl.f[i], sc);
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{c8.x, c8.y}, rq, voff_q, i * (int)a.ld_q, 0);
        }
        if (t == 0) a.s[g * a.stride_sg + ct * a.ld_s + rt] = sc.s;
    }
    if (TRANSPOSE) {
        uint8_t* const qt = MODE == kQ128Both ? a.qt + g * a.stride_qtg : a.q + g * a.stride_qg;
        float* const st = MODE == kQ128Both ? a.st + g * a.stride_stg : a.s + g * a.stride_sg;
        const int64_t ld_qt = MODE == kQ128Both ? a.ld_qt : a.ld_q;
        const int64_t ld_st = MODE == kQ128Both ? a.ld_st : a.ld_s;
        Scale scs[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) scs[j] = sc;
        uint2 codes[8];
        col_codes(tl, scs, codes);
        if (t == 0) st[rt * ld_st + ct] = sc.s;
        store_transposed(tr_lds, codes, tr, tc, qt + c0 * ld_qt + r0, ld_qt);
    }
}

template <int MODE>
__global__ __launch_bounds__(kThreads) void quant_128x128_kernel(Quant128Args a) {
    constexpr bool TRANSPOSE = MODE != kQ128Rows;
    __shared__ float s_wmax[2][4];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[TRANSPOSE ? 2 : 1][TRANSPOSE ? kTile * kTile : 16];

    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int wave = t >> 6;
    const int64_t per_g = a.row_tiles * a.col_tiles;
    const int64_t ntiles = a.G * per_g;

    auto coords = [&](int64_t tl_id, int64_t& g, int64_t& rt, int64_t& ct) {
        g = tl_id / per_g;
        const int64_t rem = tl_id % per_g;
        rt = rem / a.col_tiles;
        ct = rem % a.col_tiles;
    };

    int64_t tile = blockIdx.x;
    if (tile >= ntiles) return;
    const int voff_x = (8 * tr) * (int)(a.ld_x * 2) + 16 * tc;
    int64_t g, rt, ct;
    coords(tile, g, rt, ct);
    Raw raw;
    load_raw(a.x + g * a.stride_xg, a.ld_x, rt * kTile, ct * kTile, a.R, voff_x, raw);

    for (int parity = 0; tile < ntiles; tile += gridDim.x, parity ^= 1) {
        coords(tile, g, rt, ct);
        TileRegs tl;
        unpack_tile(raw, tl);
        const int64_t next = tile + gridDim.x;
        if (next < ntiles) {
            int64_t ng, nrt, nct;
            coords(next, ng, nrt, nct);
            load_raw(a.x + ng * a.stride_xg, a.ld_x, nrt * kTile, nct * kTile, a.R, voff_x, raw);
        }
        quant_128_tile<MODE>(a, g, rt, ct, tl, s_wmax[parity], s_tr[TRANSPOSE ? parity : 0], t, tr, tc, wave);
    }
}

// The forward operands of a linear layer in one launch: workgroups
// [0, tiles_w) take the 128x128 tiles of the weights w (both layouts, as
// quant_128x128_kernel<kQ128Both>), the rest the 128x128 tiles of x, whose
// rows and transposed columns are quantized 1x128 (as quant_1x128_kernel).
// One workgroup per tile (a grid-stride loop covers the rest if the grid is
// capped), so the two passes share one ramp-up and one tail.
__global__ __launch_bounds__(kThreads, 4) void quant_pair_kernel(Quant1x128Args xa, Quant128Args wa) {
    __shared__ float s_colmax[4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[kTile * kTile];

    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int wave = t >> 6;
    const int64_t per_g = wa.row_tiles * wa.col_tiles;
    const int64_t tiles_w = wa.G * per_g;
    const int64_t ntiles = tiles_w + ((xa.R + kTile - 1) / kTile) * xa.col_tiles;
    for (int64_t tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
        Raw raw;
        TileRegs tl;
        if (tile < tiles_w) {
            const int64_t g = tile / per_g, rem = tile % per_g;
            const int64_t rt = rem / wa.col_tiles, ct = rem % wa.col_tiles;
            load_raw(wa.x + g * wa.stride_xg, wa.ld_x, rt * kTile, ct * kTile, wa.R,
                     (8 * tr) * (int)(wa.ld_x * 2) + 16 * tc, raw);
            unpack_tile(raw, tl);
            quant_128_tile<kQ128Both>(wa, g, rt, ct, tl, s_colmax[0], s_tr, t, tr, tc, wave);
        } else {
            const int64_t xt = tile - tiles_w;
            const int64_t r0 = (xt / xa.col_tiles) * kTile, c0 = (xt % xa.col_tiles) * kTile;
            const int64_t rows = (xa.R - r0) < kTile ? (xa.R - r0) : kTile;
            load_raw(xa.x, xa.ld_x, r0, c0, xa.R, (8 * tr) * (int)(xa.ld_x * 2) + 16 * tc, raw);
            unpack_tile(raw, tl);
            quant_tile_rows(tl, rows, xa.q_row + r0 * xa.ld_qr + c0, xa.ld_qr,
                            xa.s_row + (c0 / kTile) * xa.ld_sr + r0, tr, tc);
            quant_tile_cols(tl, xa.q_col + c0 * xa.ld_qc + r0, xa.ld_qc, xa.s_col + (r0 / kTile) * xa.ld_sc + c0,
                            s_colmax, s_tr, tr, tc, wave);
        }
        if (tile + gridDim.x < ntiles) __syncthreads();  // LDS reused by the next tile
    }
}

// Persistent grid: as many workgroups as fit on the device at once (per the
// kernel's occupancy), never more than the tiles.  A problem of at least 2
// such grids' worth of tiles launches one workgroup per tile instead (the
// tile loop then runs once and never prefetches): every quantizer runs
// 4-15 % faster that way from there up to the MoE sizes (likely because
// in-order dispatch keeps the tiles in flight within one contiguous window
// of rows, where persistent workgroups drift apart), while a smaller problem
// (the 4096 x 4096 weight pass: 1024 tiles) was 12 % slower and stays
// persistent.
template <typename K>
int64_t persistent_blocks(K kernel, int64_t tiles) {
    const DeviceFit fit = device_fit(reinterpret_cast<const void*>(kernel), kThreads, 2);
    const int64_t cap = (int64_t)fit.cus * fit.per_cu;
    // (capped at 2^23 workgroups, 2^31 threads; the grid-stride loop takes the rest)
    constexpr int64_t kMaxBlocks = (int64_t)1 << 23;
    if (tiles >= 2 * cap) return tiles < kMaxBlocks ? tiles : kMaxBlocks;
    return tiles < cap ? tiles : cap;
}

}  // namespace

template <typename K, typename A>
hipError_t launch_persistent(K kernel, const A& a, int64_t tiles, hipStream_t stream) {
    dim3 grid((unsigned)persistent_blocks(kernel, tiles)), block(kThreads);
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, a);
    return hipGetLastError();
}

// persistent_blocks' choice between the two forms of a kernel: `one` (no
// prefetch) when the grid is one workgroup per tile, `persist` otherwise.
template <typename K1, typename KP, typename A>
hipError_t launch_one_or_persistent(K1 one, KP persist, const A& a, int64_t tiles, hipStream_t stream) {
    const int64_t blocks = persistent_blocks(persist, tiles);
    dim3 block(kThreads);
    if (blocks == tiles) {
        hipLaunchKernelGGL(one, dim3((unsigned)blocks), block, 0, stream, a);
    } else {
        hipLaunchKernelGGL(persist, dim3((unsigned)blocks), block, 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_quant_1x128(const Quant1x128Args& a, bool row, bool col, bool swiglu, hipStream_t stream) {
    const int64_t tiles = ((a.R + kTile - 1) / kTile) * a.col_tiles;
    if (tiles == 0) return hipSuccess;
#define BS_Q1X128(R, C, S) \
    launch_one_or_persistent(quant_1x128_kernel<R, C, S, true>, quant_1x128_kernel<R, C, S, false>, a, tiles, stream)
    if (swiglu) {
        if (row && col) return BS_Q1X128(true, true, true);
        if (row) return BS_Q1X128(true, false, true);
        return BS_Q1X128(false, true, true);
    }
    if (row && col) return BS_Q1X128(true, true, false);
    if (row) return BS_Q1X128(true, false, false);
    return BS_Q1X128(false, true, false);
#undef BS_Q1X128
}

hipError_t launch_swiglu_bwd_quant(const SwigluBwdArgs& a, bool row, bool col, hipStream_t stream) {
    const int64_t tiles = ((a.R + kTile - 1) / kTile) * a.col_tiles;
    if (tiles == 0) return hipSuccess;
    if (row && col) return launch_persistent(swiglu_bwd_quant_kernel<true, true>, a, tiles, stream);
    if (row) return launch_persistent(swiglu_bwd_quant_kernel<true, false>, a, tiles, stream);
    return launch_persistent(swiglu_bwd_quant_kernel<false, true>, a, tiles, stream);
}

hipError_t launch_mx_quant(const MxQuantArgs& a, bool row, bool col, hipStream_t stream) {
    const int64_t tiles = ((a.R + kTile - 1) / kTile) * a.col_tiles;
    if (tiles == 0) return hipSuccess;
    if (row && col) return launch_persistent(mx_quant_kernel<true, true>, a, tiles, stream);
    if (row) return launch_persistent(mx_quant_kernel<true, false>, a, tiles, stream);
    return launch_persistent(mx_quant_kernel<false, true>, a, tiles, stream);
}

hipError_t launch_quant_pair(const Quant1x128Args& xa, const Quant128Args& wa, hipStream_t stream) {
    const int64_t tiles = wa.G * wa.row_tiles * wa.col_tiles + ((xa.R + kTile - 1) / kTile) * xa.col_tiles;
    if (tiles == 0) return hipSuccess;
    constexpr int64_t kMaxBlocks = (int64_t)1 << 23;
    hipLaunchKernelGGL(quant_pair_kernel, dim3((unsigned)(tiles < kMaxBlocks ? tiles : kMaxBlocks)),
                       dim3(kThreads), 0, stream, xa, wa);
    return hipGetLastError();
}

hipError_t launch_quant_128x128(const Quant128Args& a, Quant128Mode mode, hipStream_t stream) {
    const int64_t tiles = a.G * a.row_tiles * a.col_tiles;
    if (tiles == 0) return hipSuccess;
    if (mode == kQ128Both) return launch_persistent(quant_128x128_kernel<kQ128Both>, a, tiles, stream);
    if (mode == kQ128Transposed) return launch_persistent(quant_128x128_kernel<kQ128Transposed>, a, tiles, stream);
    return launch_persistent(quant_128x128_kernel<kQ128Rows>, a, tiles, stream);
}

}  // namespace bs
