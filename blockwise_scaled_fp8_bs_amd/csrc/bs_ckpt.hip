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
//
// At 16384 x 8192 the forward takes 225 us in a step (1.10 GB, 4.9 TB/s: HBM),
// the backward 279 (3.9 TB/s; 314 with a wave less on each SIMD): 67 vector
// instructions an element, 238 us at 2.2 GHz, of them 26 the two quantizations
// of da and of db, about 19 the gradient and 9 the proof that its rounding is
// certain.
#include "bs_norm.h"
#include "bs_tile.h"

namespace bs {

namespace {

// ---- elements that the fp32 path leaves undecided ----
// A thread notes them in a 64-bit mask over its 8x8 block.  Their float64
// values are computed for one element of every lane at a time; putting them
// in place is a lane after another, so that the word's index is uniform: the
// block stays in registers, where a uniform index is an indexed move, and an
// element costs a few instructions.  (A blend of all 32 words by a per-lane
// index costs 128.)
typedef uint32_t Packed __attribute__((ext_vector_type(32)));  // word 4 i + j / 2: row i, columns j, j + 1 (bf16)

// Conditions on the wave's elements as 64-bit lane masks in scalar registers,
// combined there: as per-lane booleans they come back through a select and a
// compare when they are collected.  (The comparisons of the checks below run
// with every lane of the wave active.)
enum Cmp { kLess = 12, kGreaterEq = 11, kLessEq = 13, kNotEq = 14, kLessEqU = 37 };  // floats: or unordered
template <Cmp C>
__device__ __forceinline__ uint64_t lanes_where(float x, float y) {
    return __builtin_amdgcn_fcmpf(x, y, C);
}

// Shifts the mask left by one with the lane's bit of `lanes` as its lowest.
__device__ __forceinline__ void mark(uint32_t& m, uint64_t lanes) {
    uint64_t carry;
    asm("v_addc_co_u32_e64 %0, %1, %0, %0, %2" : "+v"(m), "=s"(carry) : "s"(lanes));
}

// Two values to a word of bf16 in one instruction.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

__device__ __forceinline__ void pack_row(Packed& p, int i, const float* f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) p[4 * i + j] = pack2(f[2 * j], f[2 * j + 1]);
}
__device__ __forceinline__ void unpack_packed(const Packed& p, TileRegs& t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack8(make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]), t.f[i]);
}

// Takes an element off a mask that is not empty.
__device__ __forceinline__ int next_marked(uint32_t& m0, uint32_t& m1) {
    const bool first = m0 != 0;
    const int bit = __builtin_clz(first ? m0 : m1);
    (first ? m0 : m1) &= ~(0x80000000u >> bit);
    return (first ? 0 : 32) + bit;
}

// value(e) gives element e's bf16 value (as a float).
template <typename F>
__device__ __forceinline__ void redo_marked(uint32_t m0, uint32_t m1, Packed& block, F&& value) {
    while (uint64_t lanes = __ballot((m0 | m1) != 0)) {
        int e = 0;
        float v = 0.f;
        if ((m0 | m1) != 0) {
            e = next_marked(m0, m1);
            v = value(e);
        }
        const uint32_t h = __float_as_uint(v) >> 16, put = h | (h << 16);
        const int lane = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        while (lanes != 0) {
            const int from = __builtin_ctzll(lanes);
            lanes &= lanes - 1;
            const int w = __builtin_amdgcn_readlane(e, from) >> 1;
            const uint32_t mask32 = lane == from ? ((e & 1) ? 0xFFFF0000u : 0xFFFFu) : 0u;
            block[w] = (put & mask32) | (block[w] & ~mask32);
        }
    }
}

// Two blocks at once (da and db, whose indexed forms would not fit beside one
// another): element e of each by blends, the masks of a row's four words
// shared by the rows and by both blocks.
__device__ __forceinline__ uint32_t blend(uint32_t mask, uint32_t put, uint32_t word) {
    return (put & mask) | (word & ~mask);
}
__device__ __forceinline__ void set_pair(Raw& x, Raw& y, int e, float vx, float vy) {
    const uint32_t hx = __float_as_uint(vx) >> 16, hy = __float_as_uint(vy) >> 16;
    const uint32_t px = hx | (hx << 16), py = hy | (hy << 16);
    const uint32_t field = (e & 1) ? 0xFFFF0000u : 0xFFFFu, w = ((uint32_t)e >> 1) & 3u, row = (uint32_t)e >> 3;
    const uint32_t k0 = w == 0 ? field : 0u, k1 = w == 1 ? field : 0u, k2 = w == 2 ? field : 0u, k3 = w == 3 ? field : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool at = row == (uint32_t)i;
        const uint32_t m0 = at ? k0 : 0u, m1 = at ? k1 : 0u, m2 = at ? k2 : 0u, m3 = at ? k3 : 0u;
        x.v[i] = make_uint4(blend(m0, px, x.v[i].x), blend(m1, px, x.v[i].y), blend(m2, px, x.v[i].z), blend(m3, px, x.v[i].w));
        y.v[i] = make_uint4(blend(m0, py, y.v[i].x), blend(m1, py, y.v[i].y), blend(m2, py, y.v[i].z), blend(m3, py, y.v[i].w));
    }
}

// exp(-a) in fp32: 2^ph by the hardware, ph = -a log2(e) rounded, times 1 + d
// with d = -a - ph ln 2, what that rounding left out (ln 2 in two parts).  As
// exp_neg in five instructions instead of six; a below 2.3e38, where ph is finite.
__device__ __forceinline__ float exp_minus(float a) {
    const float ph = -a * kLog2e;
    const float e = __builtin_amdgcn_exp2f(ph);
    const float d = __builtin_fmaf(ph, 1.90465421e-9f, __builtin_fmaf(-ph, kLn2, -a));
    return __builtin_fmaf(e, d, e);
}

// Windows, in fp32 ulps around a bf16 rounding tie, inside which a value is
// redone.  With u = 2^-24: exp_minus errs by 3.2 u (the hardware exponential's
// 2 u and an fma), s = rcp(1 + e) by 3.2 + 1 + 2 u, e s by 7.2 u, products by
// 1 u more each, so da by 10.2 u + 7.2 u |a (1 - s)| / |t|, db and h by 8.2 u;
// k u of a value is less than k of its ulps.
constexpr float kWindowDa = 11.0f, kWindowDaT = 8.0f;
constexpr uint32_t kWindow1 = 9;
// An h or db that overflows fp32 is over bf16's largest value too, by more than
// those errors, and is the infinity that the float64 value rounds to.
constexpr float kSafe = 7.9e-31f;  // 2^-100

// |low half-word of r - 0x8000| <= kWindow1
__device__ __forceinline__ uint64_t near_tie(float r) {
    return __builtin_amdgcn_uicmp((uint32_t)(uint16_t)(__float_as_uint(r) - (0x8000u - kWindow1)), 2 * kWindow1, kLessEqU);
}

// h = silu(a) b in fp32 and the lanes where its bf16 rounding is not certain:
// as swiglu_fast, with the window above.
__device__ __forceinline__ float gate_h(float a, float b, uint64_t& redo) {
    const float silu = a * __builtin_amdgcn_rcpf(1.0f + exp_minus(a));
    const float r = silu * b;
    redo = lanes_where<kLessEq>(a, -69.0f) |
           (lanes_where<kNotEq>(silu, 0.0f) & lanes_where<kLess>(fabsf(silu), kMinNormal)) | near_tie(r);
    return r;
}

// da and db in fp32 and the lanes where one of their roundings is not certain.
// |da| >= 2^-100 leaves no factor of it below the normal range (|t| < 1.1, s <
// 1), so one comparison stands for theirs; a checkpointed a is 0 or over
// 2^-9 1e-12 / 448, so silu(a) is 0 or normal.  Where exp_minus ends (2.3e38)
// it is NaN, which da's checks find.
template <bool DA, bool DB>
__device__ __forceinline__ void gate_grad(float a, float b, float dh, float& da, float& db, uint64_t& redo) {
    const float e = exp_minus(a);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    redo = lanes_where<kLessEq>(a, -69.0f);
    if (!DA) redo |= lanes_where<kGreaterEq>(a, 2e38f);
    if (DA) {
        const float an = a * (e * s);  // a (1 - s)
        const float t = 1.0f + an;
        const float p1 = dh * b;
        da = p1 * s * t;
        const float mag = fabsf(da);
        redo |= lanes_where<kNotEq>(p1, 0.0f) &
                (lanes_where<kLess>(mag, kSafe) | lanes_where<kGreaterEq>(mag, __builtin_inff()));
        redo |= lanes_where<kLessEq>((tie_distance(da) - kWindowDa) * fabsf(t), kWindowDaT * fabsf(an));
    }
    if (DB) {
        db = dh * (a * s);
        redo |= near_tie(db);
    }
}

// 1x128 codes of row i of a thread's block (columns 8 tc .. +7 of the tile)
// to q, its scale where this lane is to store it (see quant_tile_rows).
__device__ __forceinline__ void quant_row(const float* f, int i, __amdgpu_buffer_rsrc_t rq, int voff, int ld, int tc,
                                          float& my_scale) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
    const Scale sc = block_scale(__uint_as_float(row16_max(__float_as_uint(m))));
    const uint2 qv = quant8(f, sc);
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{qv.x, qv.y}, rq, voff, i * ld, 0);
    if ((tc & 7) == i) my_scale = sc.s;
}

// ---- passes of few tiles ----
// One workgroup does what a tile needs where there are tiles enough for the
// chip.  Up to one a compute unit each is shared by two: the forward's
// checkpoint codes and its h, the backward's da and its db, of which each
// recomputes what both need.  Forward and backward at 1152 x 640 (45 tiles):
// 10.1 and 12.9 us, whole 11.4 and 17.1; at 256 tiles 13.0 and 18.3, 14.8 and
// 19.1; at 512 19.6 and 29.5, 21.4 and 28.3.  One limit for both, where the
// backward's gain ends; the forward's reaches further.
enum Part { kFirst = 0, kSecond = 1, kBoth = 2 };

template <bool ROW, bool COL, int PART>
__device__ __forceinline__ void fwd_tile(const SwigluCkptArgs& a, float (*s_colmax)[kTile], uint8_t* s_tr) {
    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int64_t col_tiles = a.C / kTile;
    const int64_t r0 = (blockIdx.x / col_tiles) * kTile, c0 = (blockIdx.x % col_tiles) * kTile;
    const int64_t rows = (a.R - r0) < kTile ? (a.R - r0) : kTile;
    Raw ra, rb;
    Packed ph;
    load_raw(a.a, a.ld_a, r0, c0, a.R, (8 * tr) * (int)(a.ld_a * 2) + 16 * tc, ra);
    load_raw(a.b, a.ld_b, r0, c0, a.R, (8 * tr) * (int)(a.ld_b * 2) + 16 * tc, rb);
    const __amdgpu_buffer_rsrc_t ka = rsrc(a.ck + r0 * a.ld_ck + c0, rows * a.ld_ck);
    const __amdgpu_buffer_rsrc_t kb = rsrc(a.ck + r0 * a.ld_ck + a.C + c0, rows * a.ld_ck);
    const int voff_k = (8 * tr) * (int)a.ld_ck + 8 * tc;
    float sa = 0.f, sb = 0.f;
    uint32_t m[2] = {0u, 0u};
    // row by row: the checkpoint's codes of a and b, and h
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float fa[8], fb[8], g[8];
        unpack8(ra.v[i], fa);
        unpack8(rb.v[i], fb);
        if (PART != kFirst) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint64_t redo;
                g[j] = gate_h(fa[j], fb[j], redo);
                mark(m[i >> 2], redo);  // element 0 ends in bit 31
            }
        }
        if (PART != kSecond) {
            quant_row(fa, i, ka, voff_k, (int)a.ld_ck, tc, sa);
            quant_row(fb, i, kb, voff_k, (int)a.ld_ck, tc, sb);
        }
        if (PART != kFirst) pack_row(ph, i, g);
        __builtin_amdgcn_sched_barrier(0);
    }
    if (PART != kSecond && tc < 8) {  // lanes tc < 8 hold the scales of rows 8 tr + tc
        const __amdgpu_buffer_rsrc_t za = rsrc(a.s_ck + (c0 / kTile) * a.ld_sck + r0, rows * 4);
        const __amdgpu_buffer_rsrc_t zb = rsrc(a.s_ck + ((a.C + c0) / kTile) * a.ld_sck + r0, rows * 4);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sa), za, (8 * tr + tc) * 4, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sb), zb, (8 * tr + tc) * 4, 0, 0);
    }
    if (PART == kFirst) return;
    redo_marked(m[0], m[1], ph, [&](int e) {
        const int64_t r = r0 + 8 * tr + (e >> 3), c = c0 + 8 * tc + (e & 7);
        if (r >= a.R) return 0.f;  // rows past the end read as zeros, which are never marked
        return swiglu_bf16_f64(__uint_as_float((uint32_t)a.a[r * a.ld_a + c] << 16),
                               __uint_as_float((uint32_t)a.b[r * a.ld_b + c] << 16));
    });
    TileRegs tl;
    unpack_packed(ph, tl);
    if (ROW)
        quant_tile_rows(tl, rows, a.q_row + r0 * a.ld_qr + c0, a.ld_qr, a.s_row + (c0 / kTile) * a.ld_sr + r0, tr, tc);
    if (COL)
        quant_tile_cols(tl, a.q_col + c0 * a.ld_qc + r0, a.ld_qc, a.s_col + (r0 / kTile) * a.ld_sc + c0, s_colmax,
                        s_tr, tr, tc, t >> 6);
}

template <bool ROW, bool COL, bool SPLIT>
__global__ __launch_bounds__(kThreads) void swiglu_ckpt_kernel(SwigluCkptArgs a) {
    __shared__ float s_colmax[4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[COL ? kTile * kTile : 16];
    if (!SPLIT) fwd_tile<ROW, COL, kBoth>(a, s_colmax, s_tr);
    else if (blockIdx.y == 0) fwd_tile<ROW, COL, kSecond>(a, s_colmax, s_tr);
    else fwd_tile<ROW, COL, kFirst>(a, s_colmax, s_tr);
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

// One of da (kFirst) and db (kSecond) of a tile.
template <bool ROW, bool COL, int PART>
__device__ __forceinline__ void bwd_part(const SwigluBwdCkptArgs& a, float (*s_colmax)[kTile], uint8_t* s_tr) {
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
    if (PART == kFirst) load_ck(a.ck + r0 * a.ld_ck + a.C + c0, a.ld_ck, sb, rows, tr, tc, kb);
    load_raw(a.dh, a.ld_dh, r0, c0, a.R, (8 * tr) * (int)(a.ld_dh * 2) + 16 * tc, rd);
    Packed p;
    uint32_t m[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float fa[8], fb[8], fd[8], g[8];
        decode8(ka.q[i], ka.s[i], fa);
        if (PART == kFirst) decode8(kb.q[i], kb.s[i], fb);
        unpack8(rd.v[i], fd);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint64_t redo;
            float other;
            if (PART == kFirst) gate_grad<true, false>(fa[j], fb[j], fd[j], g[j], other, redo);
            else gate_grad<false, true>(fa[j], 0.f, fd[j], other, g[j], redo);
            mark(m[i >> 2], redo);
        }
        pack_row(p, i, g);
        __builtin_amdgcn_sched_barrier(0);
    }
    redo_marked(m[0], m[1], p, [&](int e) {
        const int rl = 8 * tr + (e >> 3);
        const int64_t r = r0 + rl, c = c0 + 8 * tc + (e & 7);
        if (r >= a.R) return 0.f;  // rows past the end read as zeros, which are never marked
        const float2 g = swiglu_grad_bf16_f64(decode1(a.ck[r * a.ld_ck + c], sa[rl]),
                                              decode1(a.ck[r * a.ld_ck + a.C + c], sb[rl]),
                                              __uint_as_float((uint32_t)a.dh[r * a.ld_dh + c] << 16));
        return PART == kFirst ? g.x : g.y;
    });
    const int64_t co = (PART == kFirst ? 0 : a.C) + c0;
    TileRegs tl;
    unpack_packed(p, tl);
    if (ROW)
        quant_tile_rows(tl, rows, a.q_row + r0 * a.ld_qr + co, a.ld_qr, a.s_row + (co / kTile) * a.ld_sr + r0, tr, tc);
    if (COL)
        quant_tile_cols(tl, a.q_col + co * a.ld_qc + r0, a.ld_qc, a.s_col + (r0 / kTile) * a.ld_sc + co, s_colmax,
                        s_tr, tr, tc, t >> 6);
}

template <bool ROW, bool COL>
__global__ __launch_bounds__(kThreads) void swiglu_bwd_ckpt_split_kernel(SwigluBwdCkptArgs a) {
    __shared__ float s_colmax[4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[COL ? kTile * kTile : 16];
    if (blockIdx.y == 0) bwd_part<ROW, COL, kFirst>(a, s_colmax, s_tr);
    else bwd_part<ROW, COL, kSecond>(a, s_colmax, s_tr);
}

template <bool ROW, bool COL>
__global__ __launch_bounds__(kThreads, 4) void swiglu_bwd_ckpt_kernel(SwigluBwdCkptArgs a) {
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
    Raw pd[2];  // da and db packed as bf16
    uint32_t m[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float fa[8], fb[8], fd[8], ga[8], gb[8];
        decode8(ka.q[i], ka.s[i], fa);
        decode8(kb.q[i], kb.s[i], fb);
        unpack8(rd.v[i], fd);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint64_t redo;
            gate_grad<true, true>(fa[j], fb[j], fd[j], ga[j], gb[j], redo);
            mark(m[i >> 2], redo);  // element 0 ends in bit 31
            if (j == 3) __builtin_amdgcn_sched_barrier(0);
        }
        pd[0].v[i] = make_uint4(pack2(ga[0], ga[1]), pack2(ga[2], ga[3]), pack2(ga[4], ga[5]), pack2(ga[6], ga[7]));
        pd[1].v[i] = make_uint4(pack2(gb[0], gb[1]), pack2(gb[2], gb[3]), pack2(gb[4], gb[5]), pack2(gb[6], gb[7]));
        __builtin_amdgcn_sched_barrier(0);
    }
    while ((m[0] | m[1]) != 0) {
        const int e = next_marked(m[0], m[1]);
        const int rl = 8 * tr + (e >> 3);
        const int64_t r = r0 + rl, c = c0 + 8 * tc + (e & 7);
        if (r >= a.R) continue;  // rows past the end read as zeros, which are never marked
        const float2 g = swiglu_grad_bf16_f64(decode1(a.ck[r * a.ld_ck + c], sa[rl]),
                                              decode1(a.ck[r * a.ld_ck + a.C + c], sb[rl]),
                                              __uint_as_float((uint32_t)a.dh[r * a.ld_dh + c] << 16));
        set_pair(pd[0], pd[1], e, g.x, g.y);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int64_t co = (half ? a.C : 0) + c0;
        TileRegs tl;
        unpack_tile(pd[half], tl);
        if (ROW)
            quant_tile_rows(tl, rows, a.q_row + r0 * a.ld_qr + co, a.ld_qr, a.s_row + (co / kTile) * a.ld_sr + r0, tr,
                            tc);
        if (COL)
            quant_tile_cols(tl, a.q_col + co * a.ld_qc + r0, a.ld_qc, a.s_col + (r0 / kTile) * a.ld_sc + co,
                            s_colmax[half], s_tr[half], tr, tc, t >> 6);
    }
}

}  // namespace

namespace {
// Up to one tile for each of the 256 compute units: two workgroups a tile.
bool split_tiles(const dim3& tiles) { return tiles.x <= 256; }
}  // namespace

hipError_t launch_swiglu_ckpt(const SwigluCkptArgs& a, hipStream_t stream) {
    dim3 grid((unsigned)(((a.R + kTile - 1) / kTile) * (a.C / kTile)));
    const dim3 block(kThreads);
    if (split_tiles(grid)) {
        grid.y = 2;
        if (a.q_row && a.q_col) hipLaunchKernelGGL((swiglu_ckpt_kernel<true, true, true>), grid, block, 0, stream, a);
        else if (a.q_row) hipLaunchKernelGGL((swiglu_ckpt_kernel<true, false, true>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((swiglu_ckpt_kernel<false, true, true>), grid, block, 0, stream, a);
    } else {
        if (a.q_row && a.q_col) hipLaunchKernelGGL((swiglu_ckpt_kernel<true, true, false>), grid, block, 0, stream, a);
        else if (a.q_row) hipLaunchKernelGGL((swiglu_ckpt_kernel<true, false, false>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((swiglu_ckpt_kernel<false, true, false>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_swiglu_bwd_ckpt(const SwigluBwdCkptArgs& a, hipStream_t stream) {
    dim3 grid((unsigned)(((a.R + kTile - 1) / kTile) * (a.C / kTile)));
    const dim3 block(kThreads);
    if (split_tiles(grid)) {
        grid.y = 2;
        if (a.q_row && a.q_col) hipLaunchKernelGGL((swiglu_bwd_ckpt_split_kernel<true, true>), grid, block, 0, stream, a);
        else if (a.q_row) hipLaunchKernelGGL((swiglu_bwd_ckpt_split_kernel<true, false>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((swiglu_bwd_ckpt_split_kernel<false, true>), grid, block, 0, stream, a);
    } else {
        if (a.q_row && a.q_col) hipLaunchKernelGGL((swiglu_bwd_ckpt_kernel<true, true>), grid, block, 0, stream, a);
        else if (a.q_row) hipLaunchKernelGGL((swiglu_bwd_ckpt_kernel<true, false>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((swiglu_bwd_ckpt_kernel<false, true>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace bs
