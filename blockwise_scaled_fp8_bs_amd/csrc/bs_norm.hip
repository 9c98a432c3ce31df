// Residual norms for gfx950: r = x + alpha gate (u rstd_u w_post), the norm of
// a block's output fused with its gate and scaled residual, and
// h = r rstd_r w_pre, the norm that the next block reads, quantized 1x128
// where its products want codes; and their backward pass.
//
// A row is held in registers by TP threads (64 or 256), NC chunks of 8 bf16
// each, between its load and its last use: x, u, dh and dr are read once.
// r is the float64 value of its formula rounded once to bf16, so that what
// the later passes and the oracle compute from r starts from the same bits;
// squares are summed in float64, which the largest finite bf16 row does not
// overflow.
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

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

__device__ __forceinline__ const void* gate_row(const void* gate, bool bf16, int64_t row) {
    return reinterpret_cast<const uint8_t*>(gate) + row * (bf16 ? 2 : 4);
}

// Sum over the TP threads of a row, in a fixed order; all of them get it.
// lds: 4 doubles per call in flight (TP = 256).
template <int TP>
__device__ __forceinline__ double row_sum(double v, double* lds) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
    if constexpr (TP > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    }
    return v;
}

template <int TP, int NC>
__global__ __launch_bounds__(256) void resid_norm_kernel(ResidNormArgs a) {
    __shared__ double s_sum[2][4];
    const int p = threadIdx.x % TP;
    const int64_t at = (int64_t)blockIdx.x * (256 / TP) + threadIdx.x / TP;
    const bool real = at < a.R;
    const int64_t row = real ? at : a.R - 1;

    uint4 raw[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = (int64_t)(p + i * TP) * 8;
        raw[i] = c < a.D ? *reinterpret_cast<const uint4*>(a.x + row * a.ld_x + c) : make_uint4(0, 0, 0, 0);
    }
    if (a.u != nullptr) {
        uint4 ru[NC];
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = (int64_t)(p + i * TP) * 8;
            ru[i] = c < a.D ? *reinterpret_cast<const uint4*>(a.u + row * a.ld_u + c) : make_uint4(0, 0, 0, 0);
        }
        double scale = a.alpha;
        if (a.w_post != nullptr) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float f[8];
                unpack8(ru[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)f[j], (double)f[j], ss);
            }
            ss = row_sum<TP>(ss, s_sum[0]);
            const double rstd = 1.0 / sqrt(ss / (double)a.D + (double)a.eps);
            scale *= rstd;
            if (a.rstd_u != nullptr && p == 0 && real) a.rstd_u[row] = (float)rstd;
        }
        const void* const gate =
            a.gate != nullptr ? gate_row(a.gate, a.w_bf16, row / a.rows_per_gate * a.ld_gate) : nullptr;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = (int64_t)(p + i * TP) * 8;
            if (c < a.D) {
                float fx[8], fu[8], w[8], g[8];
                unpack8(raw[i], fx);
                unpack8(ru[i], fu);
                fill8(w, 1.f);
                fill8(g, 1.f);
                if (a.w_post != nullptr) load_w(a.w_post, a.w_bf16, c, w);
                if (gate != nullptr) load_w(gate, a.w_bf16, c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const double wg = (double)w[j] * (double)g[j];
                    fx[j] = bf16_from_double(__builtin_fma(scale * wg, (double)fu[j], (double)fx[j]));
                }
                raw[i] = pack8(fx);
                if (real) *reinterpret_cast<uint4*>(a.r + row * a.ld_r + c) = raw[i];
            }
        }
    }
    if (a.w_pre == nullptr) return;
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float f[8];
        unpack8(raw[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)f[j], (double)f[j], ss);
    }
    ss = row_sum<TP>(ss, s_sum[1]);
    const float rstd = (float)(1.0 / sqrt(ss / (double)a.D + (double)a.eps));
    if (!real) return;
    if (a.rstd_r != nullptr && p == 0) a.rstd_r[row] = rstd;
    // with columns to quantize, the tile kernel below makes all codes from r and rstd_r
    const bool rows = a.q_row != nullptr && a.q_col == nullptr;
    if (a.h == nullptr && !rows) return;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = (int64_t)(p + i * TP) * 8;
        if (c < a.D) {
            float f[8], w[8];
            unpack8(raw[i], f);
            load_w(a.w_pre, a.w_bf16, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];
            if (a.h != nullptr) *reinterpret_cast<uint4*>(a.h + row * a.ld_h + c) = pack8(f);
            if (rows) {  // 16 lanes hold a block of 128 columns
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
                const Scale sc = block_scale(__uint_as_float(row16_max(__float_as_uint(m))));
                *reinterpret_cast<uint2*>(a.q_row + row * a.ld_qr + c) = quant8(f, sc);
                if ((p & 15) == 0) a.s_row[(c / kTile) * a.ld_sr + row] = sc.s;
            }
        }
    }
}

// Codes of h = r rstd_r w_pre along rows (ROW) and transposed columns: one
// 128x128 tile per workgroup, h in fp32 and never stored.
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
// the three sums of a row are taken in one exchange.  Each workgroup keeps the
// column sums of its rows (dh n, alpha gate dr' m, alpha dr' m w_post) in
// registers; norm_sum_kernel adds the workgroups' in a fixed order.
template <int TP, int NC>
__global__ __launch_bounds__(TP) void resid_norm_bwd_kernel(ResidNormBwdArgs a, NormBwdSplit sp, float* p_pre,
                                                            float* p_post, float* p_gate) {
    __shared__ float s_sum[2][3][4];
    const int p = threadIdx.x;
    const int64_t b = blockIdx.x;
    const int64_t S = a.rows_per_gate;
    int64_t seg = sp.chunks > 1 ? b / sp.chunks : b * sp.segs_per_block;
    const int64_t chunk = sp.chunks > 1 ? b % sp.chunks : 0;
    int64_t seg_end = sp.chunks > 1 ? seg + 1 : seg + sp.segs_per_block;
    if (seg_end > sp.segs) seg_end = sp.segs;
    const float inv_d = 1.f / (float)a.D;

    float acc_pre[NC][8], acc_post[NC][8], acc_gate[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        fill8(acc_pre[i], 0.f);
        fill8(acc_post[i], 0.f);
        fill8(acc_gate[i], 0.f);
    }
    int parity = 0;
    for (; seg < seg_end; ++seg) {
        const void* const gate = a.gate != nullptr ? gate_row(a.gate, a.w_bf16, seg * a.ld_gate) : nullptr;
        const int64_t lo = seg * S + chunk * sp.rows;
        const int64_t hi = sp.chunks > 1 ? (lo + sp.rows < (seg + 1) * S ? lo + sp.rows : (seg + 1) * S) : (seg + 1) * S;
        for (int64_t row = lo; row < hi; ++row) {
            uint4 rr[NC], ru[NC], rh[NC], rd[NC];
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int64_t c = (int64_t)(p + i * TP) * 8;
                const bool in = c < a.D;
                rr[i] = in && a.w_pre != nullptr ? *reinterpret_cast<const uint4*>(a.r + row * a.ld_r + c) : zero;
                rh[i] = in && a.w_pre != nullptr ? *reinterpret_cast<const uint4*>(a.dh + row * a.ld_dh + c) : zero;
                ru[i] = in && a.u != nullptr ? *reinterpret_cast<const uint4*>(a.u + row * a.ld_u + c) : zero;
                rd[i] = in && a.dr != nullptr ? *reinterpret_cast<const uint4*>(a.dr + row * a.ld_dr + c) : zero;
            }
            const float rstd_r = a.w_pre != nullptr ? a.rstd_r[row] : 0.f;
            const float rstd_u = a.w_post != nullptr ? a.rstd_u[row] : 1.f;
            float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int64_t c = (int64_t)(p + i * TP) * 8;
                if (c < a.D) {
                    float n[8], h[8], m[8], d[8], wp[8], wq[8], g[8];
                    unpack8(rr[i], n);
                    unpack8(rh[i], h);
                    unpack8(ru[i], m);
                    unpack8(rd[i], d);
                    fill8(wp, 0.f);
                    fill8(wq, 1.f);
                    fill8(g, 1.f);
                    if (a.w_pre != nullptr) load_w(a.w_pre, a.w_bf16, c, wp);
                    if (a.w_post != nullptr) load_w(a.w_post, a.w_bf16, c, wq);
                    if (gate != nullptr) load_w(gate, a.w_bf16, c, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float nn = n[j] * rstd_r, q = h[j] * wp[j];
                        s1 = __builtin_fmaf(q, nn, s1);
                        const float gm = g[j] * wq[j] * (m[j] * rstd_u);
                        s2 = __builtin_fmaf(gm, __builtin_fmaf(rstd_r, q, d[j]), s2);
                        s3 = __builtin_fmaf(gm, nn, s3);
                    }
                }
            }
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) {
                s1 += __shfl_xor(s1, s);
                s2 += __shfl_xor(s2, s);
                s3 += __shfl_xor(s3, s);
            }
            if constexpr (TP > 64) {
                float(*const ls)[4] = s_sum[parity];
                parity ^= 1;
                if ((p & 63) == 0) {
                    ls[0][p >> 6] = s1;
                    ls[1][p >> 6] = s2;
                    ls[2][p >> 6] = s3;
                }
                __syncthreads();
                s1 = (ls[0][0] + ls[0][1]) + (ls[0][2] + ls[0][3]);
                s2 = (ls[1][0] + ls[1][1]) + (ls[1][2] + ls[1][3]);
                s3 = (ls[2][0] + ls[2][1]) + (ls[2][2] + ls[2][3]);
            }
            const float c1 = s1 * inv_d;
            const float c2 = a.w_post != nullptr ? a.alpha * (s2 - rstd_r * c1 * s3) * inv_d : 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int64_t c = (int64_t)(p + i * TP) * 8;
                if (c < a.D) {
                    float n[8], h[8], m[8], d[8], wp[8], wq[8], g[8];
                    unpack8(rr[i], n);
                    unpack8(rh[i], h);
                    unpack8(ru[i], m);
                    unpack8(rd[i], d);
                    fill8(wp, 0.f);
                    fill8(wq, 1.f);
                    fill8(g, 1.f);
                    if (a.w_pre != nullptr) load_w(a.w_pre, a.w_bf16, c, wp);
                    if (a.w_post != nullptr) load_w(a.w_post, a.w_bf16, c, wq);
                    if (gate != nullptr) load_w(gate, a.w_bf16, c, g);
                    float du[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float nn = n[j] * rstd_r;
                        acc_pre[i][j] = __builtin_fmaf(h[j], nn, acc_pre[i][j]);
                        d[j] += rstd_r * __builtin_fmaf(-nn, c1, h[j] * wp[j]);
                        const float mm = m[j] * rstd_u, ad = a.alpha * d[j];
                        acc_post[i][j] = __builtin_fmaf(ad * g[j], mm, acc_post[i][j]);
                        acc_gate[i][j] = __builtin_fmaf(ad * wq[j], mm, acc_gate[i][j]);
                        du[j] = rstd_u * __builtin_fmaf(-mm, c2, ad * g[j] * wq[j]);
                    }
                    *reinterpret_cast<uint4*>(a.dx + row * a.ld_dx + c) = pack8(d);
                    if (a.du != nullptr) *reinterpret_cast<uint4*>(a.du + row * a.ld_du + c) = pack8(du);
                }
            }
        }
        if (a.gate != nullptr) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int64_t c = (int64_t)(p + i * TP) * 8;
                if (c < a.D) {
                    float4* o = reinterpret_cast<float4*>(p_gate + (seg * sp.chunks + chunk) * a.D + c);
                    o[0] = make_float4(acc_gate[i][0], acc_gate[i][1], acc_gate[i][2], acc_gate[i][3]);
                    o[1] = make_float4(acc_gate[i][4], acc_gate[i][5], acc_gate[i][6], acc_gate[i][7]);
                }
                fill8(acc_gate[i], 0.f);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = (int64_t)(p + i * TP) * 8;
        if (c < a.D) {
            if (p_pre != nullptr) {
                float4* o = reinterpret_cast<float4*>(p_pre + b * a.D + c);
                o[0] = make_float4(acc_pre[i][0], acc_pre[i][1], acc_pre[i][2], acc_pre[i][3]);
                o[1] = make_float4(acc_pre[i][4], acc_pre[i][5], acc_pre[i][6], acc_pre[i][7]);
            }
            if (p_post != nullptr) {
                float4* o = reinterpret_cast<float4*>(p_post + b * a.D + c);
                o[0] = make_float4(acc_post[i][0], acc_post[i][1], acc_post[i][2], acc_post[i][3]);
                o[1] = make_float4(acc_post[i][4], acc_post[i][5], acc_post[i][6], acc_post[i][7]);
            }
        }
    }
}

// Column sums of the workgroups' partial sums: block y = 0: dw_pre, 1:
// dw_post, 2 + s: segment s of dgate.  8 threads of 4 columns by 32 parts of
// the rows, the parts added in order.
__global__ __launch_bounds__(256) void norm_sum_kernel(const float* p_pre, float* dw_pre, const float* p_post,
                                                       float* dw_post, const float* p_gate, float* dgate, int64_t D,
                                                       int64_t blocks, int64_t chunks) {
    __shared__ double s_part[32][32];
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
    const int64_t c = (int64_t)blockIdx.x * 32 + 4 * x;
    const int64_t kind = blockIdx.y;
    const float* src = kind == 0 ? p_pre : kind == 1 ? p_post : p_gate + (kind - 2) * chunks * D;
    float* dst = kind == 0 ? dw_pre : kind == 1 ? dw_post : dgate + (kind - 2) * D;
    const int64_t n = kind < 2 ? blocks : chunks;
    if (dst == nullptr) return;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (c < D) {
        for (int64_t i = y; i < n; i += 32) {
            const float4 v = *reinterpret_cast<const float4*>(src + i * D + c);
            s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s_part[y][4 * x + j] = s[j];
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x < 32 && col < D) {
        double v = 0.0;
        for (int i = 0; i < 32; ++i) v += s_part[i][threadIdx.x];
        dst[col] = (float)v;
    }
}

template <int TP, int NC>
void norm_fwd(const ResidNormArgs& a, hipStream_t stream) {
    constexpr int RPB = 256 / TP;
    hipLaunchKernelGGL((resid_norm_kernel<TP, NC>), dim3((unsigned)((a.R + RPB - 1) / RPB)), dim3(256), 0, stream, a);
}

template <int TP, int NC>
void norm_bwd(const ResidNormBwdArgs& a, const NormBwdSplit& sp, float* pp, float* pq, float* pg, hipStream_t stream) {
    hipLaunchKernelGGL((resid_norm_bwd_kernel<TP, NC>), dim3((unsigned)sp.blocks), dim3(TP), 0, stream, a, sp, pp, pq,
                       pg);
}

}  // namespace

// Threads and chunks by the row's length: a wave alone (no barrier) up to
// 1024 columns, 256 threads beyond, the fewest chunks that hold the row.
#define BS_NORM_BY_D(CALL)                      \
    if (a.D <= 512) { CALL(64, 1); }            \
    else if (a.D <= 1024) { CALL(64, 2); }      \
    else if (a.D <= 2048) { CALL(256, 1); }     \
    else if (a.D <= 4096) { CALL(256, 2); }     \
    else if (a.D <= 6144) { CALL(256, 3); }     \
    else if (a.D <= 8192) { CALL(256, 4); }     \
    else { CALL(256, 8); }

hipError_t launch_resid_norm(const ResidNormArgs& a, hipStream_t stream) {
#define BS_CALL(TP, NC) norm_fwd<TP, NC>(a, stream)
    BS_NORM_BY_D(BS_CALL)
#undef BS_CALL
    if (a.q_col != nullptr) {
        const dim3 grid((unsigned)((a.R / kTile) * (a.D / kTile))), block(kThreads);
        if (a.q_row != nullptr) hipLaunchKernelGGL(norm_quant_kernel<true>, grid, block, 0, stream, a);
        else hipLaunchKernelGGL(norm_quant_kernel<false>, grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

NormBwdSplit norm_bwd_split(int64_t R, int64_t rows_per_gate) {
    // about 1024 workgroups, four for each CU, so that the rows of one hide
    // another's loads; a chunk never crosses a gate's segment
    const int64_t S = rows_per_gate, want = (R + 1023) / 1024;
    NormBwdSplit sp{};
    sp.segs = R / S;
    if (S > want) {
        sp.segs_per_block = 1;
        sp.chunks = (S + want - 1) / want;
        sp.rows = (S + sp.chunks - 1) / sp.chunks;
        sp.chunks = (S + sp.rows - 1) / sp.rows;
        sp.blocks = sp.segs * sp.chunks;
    } else {
        sp.segs_per_block = want / S > 0 ? want / S : 1;
        sp.chunks = 1;
        sp.rows = S;
        sp.blocks = (sp.segs + sp.segs_per_block - 1) / sp.segs_per_block;
    }
    return sp;
}

hipError_t launch_resid_norm_bwd(const ResidNormBwdArgs& a, hipStream_t stream) {
    const NormBwdSplit sp = norm_bwd_split(a.R, a.rows_per_gate);
    float* at = a.ws;
    float *pp = nullptr, *pq = nullptr, *pg = nullptr;
    if (a.dw_pre != nullptr) { pp = at; at += sp.blocks * a.D; }
    if (a.dw_post != nullptr) { pq = at; at += sp.blocks * a.D; }
    if (a.dgate != nullptr) {
        pg = sp.chunks > 1 ? at : a.dgate;  // whole segments need no second pass
    }
#define BS_CALL(TP, NC) norm_bwd<TP, NC>(a, sp, pp, pq, pg, stream)
    BS_NORM_BY_D(BS_CALL)
#undef BS_CALL
    const int64_t kinds = a.dgate != nullptr && sp.chunks > 1 ? 2 + sp.segs : 2;
    hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((a.D + 31) / 32), (unsigned)kinds), dim3(256), 0, stream, pp,
                       a.dw_pre, pq, a.dw_post, pg, a.dgate, a.D, sp.blocks, sp.chunks);
    return hipGetLastError();
}

}  // namespace bs
