// Residual norms for gfx950: r = x + alpha gate (u rstd_u w_post), the norm of
// a block's output fused with its gate and scaled residual, and
// h = r rstd_r w_pre, the norm that the next block reads, quantized 1x128
// where its products want codes; and their backward pass.
//
// Bound by HBM: each tensor of a row is read once and held in registers, in
// chunks of 8 bf16 a thread, between its load and its last use; a workgroup
// walks down consecutive rows with the parameters in registers and the next
// row's loads under way.  At 16384 rows of 5120, fp32 parameters: r and
// rstd_r from x and u 111 us (503 MB, 4.5 TB/s), h's codes along rows and
// columns from r 61 us, the backward pass 210 us (1.01 GB, 4.8 TB/s); with
// the parameters read again for every row it took 430 us.
//
// r is the float64 value of its formula rounded once to bf16, so that what
// the later passes and the oracle compute from r starts from the same bits.
// Sums of squares are exact enough for that in float64 (u), and by fours in
// fp32 for r, whose rstd errs by at most 2^-23.
#include "bs_norm.h"
#include "bs_tile.h"

namespace bs {

namespace {

// 8 parameters from column c on.
__device__ __forceinline__ void load_w(const void* p, bool bf16, int64_t c, float* f) {
    if (bf16) {
        unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + c), f);
    } else {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + c);
        const float4 a = q[0], b = q[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}

__device__ __forceinline__ void fill8(float* f, float v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v;
}

// f times 8 parameters from column c on.
__device__ __forceinline__ void mul_w(const void* p, bool bf16, int64_t c, float* f) {
    float w[8];
    load_w(p, bf16, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= w[j];
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

__device__ __forceinline__ const void* gate_row(const void* gate, bool bf16, int64_t row) {
    return reinterpret_cast<const uint8_t*>(gate) + row * (bf16 ? 2 : 4);
}

// 16 bytes of row `row` from column c on; columns past n bytes read 0 (the
// descriptor ends with the row; that of an absent tensor is empty).
__device__ __forceinline__ u32x4 load_row(const uint16_t* base, int64_t row, int64_t ld, int64_t n, int c) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc(base + row * ld, n), 2 * c, 0, 0));
}
__device__ __forceinline__ void store_row(uint16_t* base, int64_t row, int64_t ld, int64_t n, int c, uint4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{v.x, v.y, v.z, v.w}, rsrc(base + row * ld, n), 2 * c, 0, 0);
}
__device__ __forceinline__ void unpack8(u32x4 v, float* f) { bs::unpack8(make_uint4(v[0], v[1], v[2], v[3]), f); }

// One DPP step of a sum over a wave.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
    return v + __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}

// Sum over the wave, in its last lane: quads, halves of rows, rows, then row
// 0 into 1 and 2 into 3, then both into the last.
template <typename T>
__device__ __forceinline__ T wave_sum_last(T v) {
    v = dpp_add<0xB1, 0xF>(v);   // quad_perm 1,0,3,2
    v = dpp_add<0x4E, 0xF>(v);   // quad_perm 2,3,0,1
    v = dpp_add<0x141, 0xF>(v);  // row_half_mirror
    v = dpp_add<0x140, 0xF>(v);  // row_mirror
    v = dpp_add<0x142, 0xA>(v);  // row_bcast 15
    v = dpp_add<0x143, 0xC>(v);  // row_bcast 31
    return v;
}

// Sum over the workgroup in a fixed order, in every thread.  lds: 16 values,
// zeroed before the first use (waves that are not there add 0), two of them
// in turn for sums that follow one another.
template <int MAXT, typename T>
__device__ __forceinline__ T block_sum(T v, T* lds) {
    v = wave_sum_last(v);
    if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    T s = 0;
#pragma unroll
    for (int w = 0; w < (MAXT + 192) / 256 * 4; w += 4) s += (lds[w] + lds[w + 1]) + (lds[w + 2] + lds[w + 3]);
    return s;
}

// 1 / sqrt(v) in float64: the hardware's estimate and two Newton steps, in
// which infinity times 0 is NaN: the estimate of 0 (infinity) and that of
// infinity (0) stand as they are.
__device__ __forceinline__ double rsqrt64(double v) {
    const double y0 = __builtin_amdgcn_rsq(v);
    const double h = 0.5 * v;
    double y = y0 * __builtin_fma(-h * y0, y0, 1.5);
    y = y * __builtin_fma(-h * y, y, 1.5);
    return y == y ? y : y0;
}

// A workgroup has a thread for each NC chunks of 8 columns and walks down
// `per` rows: the parameters stay in registers, and a row's loads are under
// way while the one before it is worked on.
// HOLD: without it (rows of more than 8192 columns, whose chunks would not
// fit beside them) the parameters and the row are read where they are used.
template <int NC, int MAXT, bool HOLD>
__global__ __launch_bounds__(MAXT) void resid_norm_kernel(ResidNormArgs a, int64_t per) {
    __shared__ double s_sum[3][16];  // of u; of r (without a norm of u the two in turn); of r again
    const int p = threadIdx.x, TP = blockDim.x;
    const int64_t lo = (int64_t)blockIdx.x * per, hi = lo + per < a.R ? lo + per : a.R;
    const int64_t bytes = a.D * 2, b_u = a.u != nullptr ? bytes : 0;
    const bool pre = a.w_pre != nullptr, post = a.w_post != nullptr, has_u = a.u != nullptr;
    const double inv_d = 1.0 / (double)a.D, eps = (double)a.eps;
    // with columns to quantize, the tile kernel below makes all codes from r and rstd_r
    const bool rows = a.q_row != nullptr && a.q_col == nullptr;

    int col[NC];
    bool in[NC];
    float wp_held[NC][8];
    double wg_held[NC][8];  // alpha gate w_post
    auto load_wp = [&](int i, float* f) {
        fill8(f, 0.f);
        if (pre && in[i]) load_w(a.w_pre, a.w_bf16, col[i], f);
    };
    auto load_wg = [&](const void* gate, int i, double* f) {
        float w[8], g[8];
        fill8(w, 1.f);
        fill8(g, 1.f);
        if (in[i] && post) load_w(a.w_post, a.w_bf16, col[i], w);
        if (in[i] && gate != nullptr) load_w(gate, a.w_bf16, col[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (double)w[j] * (double)g[j] * (double)a.alpha;
    };
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        col[i] = (p + i * TP) * 8;
        in[i] = col[i] < a.D;
        if (HOLD) load_wp(i, wp_held[i]);
    }
    if (p < 48) (&s_sum[0][0])[p] = 0.0;
    __syncthreads();

    u32x4 cur_x[NC], cur_u[NC], next_x[NC], next_u[NC];
    auto load = [&](int64_t row, u32x4* ox, u32x4* ou) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            ox[i] = load_row(a.x, row, a.ld_x, bytes, col[i]);
            ou[i] = load_row(a.u, row, a.ld_u, b_u, col[i]);
        }
    };
    if (HOLD) load(lo, next_x, next_u);
    int64_t seg_end = lo;  // first row of the next gate segment
    const void* gate = nullptr;
    for (int64_t row = lo; row < hi; ++row) {
        if (HOLD) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                cur_x[i] = next_x[i];
                cur_u[i] = next_u[i];
            }
            if (row + 1 < hi) load(row + 1, next_x, next_u);
        } else {
            load(row, cur_x, cur_u);
        }
        if (has_u) {
            if (row == seg_end) {
                const int64_t seg = row / a.rows_per_gate;
                seg_end = (seg + 1) * a.rows_per_gate;
                if (a.gate != nullptr) gate = gate_row(a.gate, a.w_bf16, seg * a.ld_gate);
                if (HOLD && (row == lo || gate != nullptr)) {
#pragma unroll
                    for (int i = 0; i < NC; ++i) load_wg(gate, i, wg_held[i]);
                }
            }
            double rstd = 1.0;
            if (post) {
                double ss = 0.0;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float f[8];
                    unpack8(cur_u[i], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)f[j], (double)f[j], ss);
                }
                ss = block_sum<MAXT>(ss, s_sum[0]);
                rstd = rsqrt64(__builtin_fma(ss, inv_d, eps));
                if (a.rstd_u != nullptr && p == 0) a.rstd_u[row] = (float)rstd;
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float f[8], fu[8];
                double wg[8], d[8];
                unpack8(cur_x[i], f);
                unpack8(cur_u[i], fu);
                if (!HOLD) load_wg(gate, i, wg);
                // float64 to fp32 to bf16 is one rounding unless the fp32 value
                // is a tie between two bf16 ones (one in 2^16): those are redone
                uint32_t tie = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    d[j] = __builtin_fma(rstd * (HOLD ? wg_held[i][j] : wg[j]), (double)fu[j], (double)f[j]);
                    f[j] = (float)d[j];
                    tie |= (__float_as_uint(f[j]) & 0xFFFFu) == 0x8000u ? 1u : 0u;
                }
                if (tie) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = bf16_from_double(d[j]);
                }
                const uint4 v = pack8(f);
                cur_x[i] = u32x4{v.x, v.y, v.z, v.w};
                store_row(a.r, row, a.ld_r, bytes, col[i], v);
            }
        }
        if (!pre) {
            if (post) __syncthreads();  // s_sum[0] is written again in the next row
            continue;
        }
        // squares four by four in fp32 (two roundings: rstd_r errs by half of
        // them and its own, 2^-23), their sums in float64; all in float64
        // where four leave fp32's range
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float f[8];
            unpack8(cur_x[i], f);
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                ss += (double)(__builtin_fmaf(f[j], f[j], f[j + 1] * f[j + 1]) +
                               __builtin_fmaf(f[j + 2], f[j + 2], f[j + 3] * f[j + 3]));
        }
        ss = block_sum<MAXT>(ss, s_sum[post ? 1 : (int)(row & 1)]);
        if (!(ss > 1e-25 && ss < __builtin_inf())) {
            ss = 0.0;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float f[8];
                unpack8(cur_x[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)f[j], (double)f[j], ss);
            }
            ss = block_sum<MAXT>(ss, s_sum[2]);
        }
        const float rstd = (float)rsqrt64(__builtin_fma(ss, inv_d, eps));
        if (a.rstd_r != nullptr && p == 0) a.rstd_r[row] = rstd;
        if (a.h == nullptr && !rows) continue;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float f[8];
            unpack8(cur_x[i], f);
            float wp[8];
            if (!HOLD) load_wp(i, wp);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * (HOLD ? wp_held[i][j] : wp[j]);
            if (a.h != nullptr) store_row(a.h, row, a.ld_h, bytes, col[i], pack8(f));
            if (rows && in[i]) {  // 16 lanes hold a block of 128 columns
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
                const Scale sc = block_scale(__uint_as_float(row16_max(__float_as_uint(m))));
                *reinterpret_cast<uint2*>(a.q_row + row * a.ld_qr + col[i]) = quant8(f, sc);
                if ((p & 15) == 0) a.s_row[(col[i] / kTile) * a.ld_sr + row] = sc.s;
            }
        }
    }
}

// Codes of h = r rstd_r w_pre along rows (ROW) and transposed columns: one
// 128x128 tile per workgroup, h in fp32 and never stored.  Bound by HBM: at
// 16384 x 5120 60 us for both (340 MB, 5.6 TB/s).
template <bool ROW>
__global__ __launch_bounds__(kThreads) void norm_quant_kernel(ResidNormArgs a) {
    __shared__ float s_colmax[4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[kTile * kTile];
    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int64_t col_tiles = a.D / kTile;
    const int64_t r0 = (blockIdx.x / col_tiles) * kTile, c0 = (blockIdx.x % col_tiles) * kTile;
    const uint16_t* const src = a.u != nullptr ? a.r : a.x;
    const int64_t ld = a.u != nullptr ? a.ld_r : a.ld_x;
    Raw raw;
    load_raw(src, ld, r0, c0, a.R, (8 * tr) * (int)(ld * 2) + 16 * tc, raw);
    float rs[8], w[8];
    load_w(a.rstd_r, false, r0 + 8 * tr, rs);
    load_w(a.w_pre, a.w_bf16, c0 + 8 * tc, w);
    TileRegs tl;
    unpack_tile(raw, tl);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) tl.f[i][j] = tl.f[i][j] * rs[i] * w[j];
    if (ROW)
        quant_tile_rows(tl, kTile, a.q_row + r0 * a.ld_qr + c0, a.ld_qr, a.s_row + (c0 / kTile) * a.ld_sr + r0, tr,
                        tc);
    quant_tile_cols(tl, a.q_col + c0 * a.ld_qc + r0, a.ld_qc, a.s_col + (r0 / kTile) * a.ld_sc + c0, s_colmax, s_tr,
                    tr, tc, t >> 6);
}

// Backward.  With n = r rstd_r, m = u rstd_u, q = dh w_pre and
// G = alpha gate w_post:
//   dr' = dr + rstd_r (q - n mean(q n))            (dx; what flows into u's side)
//   du  = rstd_u (G dr' - m mean(G dr' m))
// mean(G dr' m) = (sum G m (dr + rstd_r q) - rstd_r mean(q n) sum G m n) / D, so
// the three sums of a row are taken in one exchange.  A workgroup has a
// thread for each NC chunks of 8 columns and walks down its rows: the
// parameters and the column sums (dh n and dr' m, of which the gradients of
// w_post and of the gate are multiples within a gate's segment) stay in
// registers, and a row's loads are under way while the one before it is
// worked on.  norm_sum_kernel adds the workgroups' sums in a fixed order.
struct NormRow {
    u32x4 r, u, h, d;
};

// HOLD: the parameters and the next row stay in registers.  Without it (rows
// of more than 8192 columns, whose two chunks a thread would not fit beside
// them) both are read where they are used, and a workgroup has one segment: at
// 16384 x 16384 1054 us (3.2 GB of tensors, 3.1 TB/s; forward r alone 413, 3.9).
template <int NC, int MAXT, bool HOLD>
__global__ __launch_bounds__(MAXT) void resid_norm_bwd_kernel(ResidNormBwdArgs a, NormBwdSplit sp, float* p_pre,
                                                              float* p_post, float* p_gate) {
    __shared__ __attribute__((aligned(16))) float s_sum[2][3][16];
    const int p = threadIdx.x, TP = blockDim.x;
    const int64_t b = blockIdx.x;
    const int64_t S = a.rows_per_gate;
    int64_t seg = sp.chunks > 1 ? b / sp.chunks : b * sp.segs_per_block;
    const int64_t chunk = sp.chunks > 1 ? b % sp.chunks : 0;
    int64_t seg_end = sp.chunks > 1 ? seg + 1 : seg + sp.segs_per_block;
    if (seg_end > sp.segs) seg_end = sp.segs;
    const float inv_d = 1.f / (float)a.D;
    const bool pre = a.w_pre != nullptr, post = a.w_post != nullptr;

    const int64_t bytes = a.D * 2, b_pre = pre ? bytes : 0, b_u = a.u != nullptr ? bytes : 0;
    const int64_t b_d = a.dr != nullptr ? bytes : 0;
    bool in[NC];
    int col[NC];
    float wp_held[NC][8], acc_pre[NC][8], acc_post[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        col[i] = (p + i * TP) * 8;
        in[i] = col[i] < a.D;
        fill8(acc_pre[i], 0.f);
        fill8(acc_post[i], 0.f);
        if (HOLD) {
            fill8(wp_held[i], 0.f);
            if (pre && in[i]) load_w(a.w_pre, a.w_bf16, col[i], wp_held[i]);
        }
    }
    // w_pre, and alpha gate w_post, of chunk i
    auto load_wp = [&](int i, float* f) {
        fill8(f, 0.f);
        if (pre && in[i]) load_w(a.w_pre, a.w_bf16, col[i], f);
    };
    auto load_g = [&](const void* gate, int i, float* f) {
        fill8(f, a.alpha);
        if (in[i] && gate != nullptr) mul_w(gate, a.w_bf16, col[i], f);
        if (in[i] && post) mul_w(a.w_post, a.w_bf16, col[i], f);
    };
    for (int i = p; i < 96; i += TP) (&s_sum[0][0][0])[i] = 0.f;  // waves that are not there add 0
    __syncthreads();
    auto load = [&](int64_t row, NormRow* o) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            o[i].r = load_row(a.r, row, a.ld_r, b_pre, col[i]);
            o[i].h = load_row(a.dh, row, a.ld_dh, b_pre, col[i]);
            o[i].u = load_row(a.u, row, a.ld_u, b_u, col[i]);
            o[i].d = load_row(a.dr, row, a.ld_dr, b_d, col[i]);
        }
    };
    int parity = 0;
    for (; seg < seg_end; ++seg) {
        const void* const gate = a.gate != nullptr ? gate_row(a.gate, a.w_bf16, seg * a.ld_gate) : nullptr;
        const int64_t lo = seg * S + chunk * sp.rows;
        const int64_t hi = sp.chunks > 1 ? (lo + sp.rows < (seg + 1) * S ? lo + sp.rows : (seg + 1) * S) : (seg + 1) * S;
        float g_held[NC][8], acc_m[NC][8];  // alpha gate w_post; sum of dr' m
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            fill8(acc_m[i], 0.f);
            if (HOLD) load_g(gate, i, g_held[i]);
        }
        NormRow cur[NC], next[NC];
        if (HOLD) load(lo, next);
        for (int64_t row = lo; row < hi; ++row) {
            if (HOLD) {
#pragma unroll
                for (int i = 0; i < NC; ++i) cur[i] = next[i];
            } else {
                load(row, cur);
            }
            const float rstd_r = pre ? a.rstd_r[row] : 0.f;
            const float rstd_u = post ? a.rstd_u[row] : 1.f;
            if (HOLD && row + 1 < hi) load(row + 1, next);
            float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float n[8], h[8], m[8], d[8];
                unpack8(cur[i].r, n);
                unpack8(cur[i].h, h);
                unpack8(cur[i].u, m);
                unpack8(cur[i].d, d);
                float wp[8], G[8];
                if (!HOLD) load_wp(i, wp);
                if (!HOLD) load_g(gate, i, G);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float nn = n[j] * rstd_r, q = h[j] * (HOLD ? wp_held[i][j] : wp[j]);
                    s1 = __builtin_fmaf(q, nn, s1);
                    const float gm = (HOLD ? g_held[i][j] : G[j]) * (m[j] * rstd_u);
                    s2 = __builtin_fmaf(gm, __builtin_fmaf(rstd_r, q, d[j]), s2);
                    s3 = __builtin_fmaf(gm, nn, s3);
                }
            }
            s1 = wave_sum_last(s1);
            s2 = wave_sum_last(s2);
            s3 = wave_sum_last(s3);
            float(*const ls)[16] = s_sum[parity];
            parity ^= 1;
            if ((p & 63) == 63) {
                ls[0][p >> 6] = s1;
                ls[1][p >> 6] = s2;
                ls[2][p >> 6] = s3;
            }
            __syncthreads();
            float t3[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                t3[k] = 0.f;
#pragma unroll
                for (int w = 0; w < (MAXT + 192) / 256 * 4; w += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(&ls[k][w]);
                    t3[k] += (v.x + v.y) + (v.z + v.w);
                }
            }
            const float c1 = t3[0] * inv_d;
            const float c2 = post ? (t3[1] - rstd_r * c1 * t3[2]) * inv_d : 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float n[8], h[8], m[8], d[8], du[8];
                unpack8(cur[i].r, n);
                unpack8(cur[i].h, h);
                unpack8(cur[i].u, m);
                unpack8(cur[i].d, d);
                float wp[8], G[8];
                if (!HOLD) load_wp(i, wp);
                if (!HOLD) load_g(gate, i, G);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float nn = n[j] * rstd_r;
                    acc_pre[i][j] = __builtin_fmaf(h[j], nn, acc_pre[i][j]);
                    d[j] += rstd_r * __builtin_fmaf(-nn, c1, h[j] * (HOLD ? wp_held[i][j] : wp[j]));
                    const float mm = m[j] * rstd_u;
                    acc_m[i][j] = __builtin_fmaf(d[j], mm, acc_m[i][j]);
                    du[j] = rstd_u * __builtin_fmaf(-mm, c2, (HOLD ? g_held[i][j] : G[j]) * d[j]);
                }
                store_row(a.dx, row, a.ld_dx, bytes, col[i], pack8(d));
                store_row(a.du, row, a.ld_du, b_u, col[i], pack8(du));
            }
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (!in[i]) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc_m[i][j] *= a.alpha;
            if (p_gate != nullptr) {
                float g[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = acc_m[i][j];
                if (post) mul_w(a.w_post, a.w_bf16, col[i], g);
                float4* o = reinterpret_cast<float4*>(p_gate + (seg * sp.chunks + chunk) * a.D + col[i]);
                o[0] = make_float4(g[0], g[1], g[2], g[3]);
                o[1] = make_float4(g[4], g[5], g[6], g[7]);
            }
            if (gate != nullptr) mul_w(gate, a.w_bf16, col[i], acc_m[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc_post[i][j] = HOLD ? acc_post[i][j] + acc_m[i][j] : acc_m[i][j];
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if (!in[i]) continue;
        if (p_pre != nullptr) {
            float4* o = reinterpret_cast<float4*>(p_pre + b * a.D + col[i]);
            o[0] = make_float4(acc_pre[i][0], acc_pre[i][1], acc_pre[i][2], acc_pre[i][3]);
            o[1] = make_float4(acc_pre[i][4], acc_pre[i][5], acc_pre[i][6], acc_pre[i][7]);
        }
        if (p_post != nullptr) {
            float4* o = reinterpret_cast<float4*>(p_post + b * a.D + col[i]);
            o[0] = make_float4(acc_post[i][0], acc_post[i][1], acc_post[i][2], acc_post[i][3]);
            o[1] = make_float4(acc_post[i][4], acc_post[i][5], acc_post[i][6], acc_post[i][7]);
        }
    }
}

// Column sums of the workgroups' partial sums: block y = 0: dw_pre, 1:
// dw_post, beyond: 4 segments of dgate each.  A column's rows are summed in
// 128 parts (of dgate, which has few rows a segment, in 32), and the parts
// added in order.  Latency: 4 us for 256 sums of 5120, 6 for 1024 of 1024 (12
// in 32 parts), 9 for 2048 of 512 (22).
constexpr int kSumParts = 128, kSumSegs = 4;
__global__ __launch_bounds__(8 * kSumParts) void norm_sum_kernel(const float* p_pre, float* dw_pre,
                                                                 const float* p_post, float* dw_post,
                                                                 const float* p_gate, float* dgate, int64_t D,
                                                                 int64_t blocks, int64_t chunks, int64_t segs) {
    __shared__ double s_part[kSumParts][32];
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
    const int64_t c = (int64_t)blockIdx.x * 32 + 4 * x;
    const bool gate = blockIdx.y >= 2;
    const int64_t seg0 = gate ? (int64_t)(blockIdx.y - 2) * kSumSegs : 0;
    float* const dst = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
    if (dst == nullptr) return;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    // rows first, first + step, ... of src: four loads under way at a time, the last row in the place of those past it
    const auto add = [&](const float* src, int64_t first, int64_t step, int64_t n) {
        for (int64_t i = first; i < n; i += 4 * step) {
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t at = i + k * step < n ? i + k * step : n - 1;
                v[k] = *reinterpret_cast<const float4*>(src + at * D + c);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (i + k * step >= n) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                s[0] += v[k].x; s[1] += v[k].y; s[2] += v[k].z; s[3] += v[k].w;
            }
        }
    };
    if (c < D && gate) {
        constexpr int kParts = kSumParts / kSumSegs;
        const int64_t seg = seg0 + y / kParts;
        if (seg < segs) add(p_gate + seg * chunks * D, y % kParts, kParts, chunks);
    } else if (c < D) {
        add(blockIdx.y == 0 ? p_pre : p_post, y, kSumParts, blocks);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s_part[y][4 * x + j] = s[j];
    __syncthreads();
    const int q = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + q;
    if (!gate) {  // 32 columns by 32 groups of 4 parts first
        const double four = ((s_part[4 * g][q] + s_part[4 * g + 1][q]) + s_part[4 * g + 2][q]) + s_part[4 * g + 3][q];
        __syncthreads();
        s_part[g][q] = four;
        __syncthreads();
    }
    if (g < (gate ? kSumSegs : 1) && col < D && seg0 + g < (gate ? segs : 1)) {
        double v = 0.0;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) v += s_part[32 * g + i][q];
        dst[(seg0 + g) * D + col] = (float)v;
    }
}
static_assert(kSumParts / kSumSegs == 32 && kSumParts / 4 == 32, "32 sums are left for the last step");

// Threads of a workgroup: the chunks of a row over NC, in whole waves.
template <int NC>
unsigned norm_threads(int64_t D) {
    return (unsigned)((D / 8 + 64 * NC - 1) / (64 * NC) * 64);
}

template <int NC, int MAXT>
void norm_fwd(const ResidNormArgs& a, hipStream_t stream) {
    const unsigned threads = norm_threads<NC>(a.D);
    // enough workgroups for 32 waves of one chunk on each of 256 CUs, so that a
    // CU has several to change between and each still walks down many rows
    const int64_t waves = NC * threads / 64, blocks = 256 * (waves < 32 ? 32 / waves : 1);
    constexpr bool kHold = NC * MAXT <= 1024;
    const int64_t per = kHold ? (a.R + blocks - 1) / blocks : 1;
    hipLaunchKernelGGL((resid_norm_kernel<NC, MAXT, kHold>), dim3((unsigned)((a.R + per - 1) / per)),
                       dim3(threads), 0, stream, a, per);
}

template <int NC, int MAXT>
void norm_bwd(const ResidNormBwdArgs& a, const NormBwdSplit& sp, float* pp, float* pq, float* pg, hipStream_t stream) {
    hipLaunchKernelGGL((resid_norm_bwd_kernel<NC, MAXT, NC == 1>), dim3((unsigned)sp.blocks),
                       dim3(norm_threads<NC>(a.D)), 0, stream, a, sp, pp, pq, pg);
}

}  // namespace

hipError_t launch_resid_norm(const ResidNormArgs& a, hipStream_t stream) {
    // D = 5120 at 16384 rows, r alone: 111 us in three chunks, 118 in one, 129 in two (640 threads
    // are ten waves on four SIMDs, and a second workgroup of them does not fit beside the first); at
    // 4104 columns 98, 120 and 126, at 6144 129, 125 and 125, with h written too 175, 175 and 176
    if (a.D <= 2048) norm_fwd<1, 256>(a, stream);
    else if (a.D <= 4096) norm_fwd<1, 512>(a, stream);
    else if (a.D <= 6144) norm_fwd<3, 256>(a, stream);
    else if (a.D <= 8192) norm_fwd<1, 1024>(a, stream);
    else norm_fwd<2, 1024>(a, stream);
    if (a.q_col != nullptr) {
        const dim3 grid((unsigned)((a.R / kTile) * (a.D / kTile))), block(kThreads);
        if (a.q_row != nullptr) hipLaunchKernelGGL(norm_quant_kernel<true>, grid, block, 0, stream, a);
        else hipLaunchKernelGGL(norm_quant_kernel<false>, grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

NormBwdSplit norm_bwd_split(int64_t R, int64_t D, int64_t rows_per_gate) {
    // workgroups for 8 waves on each of 256 CUs (at 16384 rows of 1024 columns:
    // 48 us, 62 with 2 waves; of 4096: 165 us, 175 with 16; more of them write
    // more partial sums); a chunk never crosses a gate's segment
    const int64_t waves = (D + 511) / 512;
    int64_t blocks = 256 * (waves < 8 ? 8 / waves : 1);
    // where that leaves less than 4 rows each, half of them: 2048 rows of 512
    // 14.6 us (19.4), 1000 of 1024 15.0 (17.6), 693 of 2048 15.1 (16.5)
    if (R < 4 * blocks && waves < 8) blocks /= 2;
    const int64_t S = rows_per_gate, want = (R + blocks - 1) / blocks;
    NormBwdSplit sp{};
    sp.segs = R / S;
    if (S > want) {
        sp.segs_per_block = 1;
        sp.chunks = (S + want - 1) / want;
        sp.rows = (S + sp.chunks - 1) / sp.chunks;
        sp.chunks = (S + sp.rows - 1) / sp.rows;
        sp.blocks = sp.segs * sp.chunks;
    } else {
        sp.segs_per_block = want / S > 0 && D <= 8192 ? want / S : 1;
        sp.chunks = 1;
        sp.rows = S;
        sp.blocks = (sp.segs + sp.segs_per_block - 1) / sp.segs_per_block;
    }
    return sp;
}

hipError_t launch_resid_norm_bwd(const ResidNormBwdArgs& a, hipStream_t stream) {
    const NormBwdSplit sp = norm_bwd_split(a.R, a.D, a.rows_per_gate);
    float* at = a.ws;
    float *pp = nullptr, *pq = nullptr, *pg = nullptr;
    if (a.dw_pre != nullptr) { pp = at; at += sp.blocks * a.D; }
    if (a.dw_post != nullptr) { pq = at; at += sp.blocks * a.D; }
    if (a.dgate != nullptr) {
        pg = sp.chunks > 1 ? at : a.dgate;  // whole segments need no second pass
    }
    // the bound on the threads sets how many registers one may take
    if (a.D <= 2048) norm_bwd<1, 256>(a, sp, pp, pq, pg, stream);
    else if (a.D <= 4096) norm_bwd<1, 512>(a, sp, pp, pq, pg, stream);
    else if (a.D <= 6144) norm_bwd<1, 768>(a, sp, pp, pq, pg, stream);
    else if (a.D <= 8192) norm_bwd<1, 1024>(a, sp, pp, pq, pg, stream);
    else norm_bwd<2, 1024>(a, sp, pp, pq, pg, stream);
    const int64_t kinds = a.dgate != nullptr && sp.chunks > 1 ? 2 + (sp.segs + kSumSegs - 1) / kSumSegs : 2;
    hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((a.D + 31) / 32), (unsigned)kinds), dim3(8 * kSumParts), 0, stream, pp,
                       a.dw_pre, pq, a.dw_post, pg, a.dgate, a.D, sp.blocks, sp.chunks, sp.segs);
    return hipGetLastError();
}

}  // namespace bs
