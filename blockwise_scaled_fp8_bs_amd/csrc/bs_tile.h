// The 128x128 tile of the quantizer kernels: loads with bounds, row and column
// blocks, transposed stores through LDS, and the gated activation's
// arithmetic.  Shared by the kernels that quantize what they compute
// (bs_quant.hip, bs_moe.hip, bs_norm.hip, bs_ckpt.hip).  gfx950 only.
//
// A tile is owned by 256 threads (4 wave64s); thread t holds an 8x8
// sub-block: rows 8*(t/16) .. +7 and columns 8*(t%16) .. +7.
#pragma once

#include "bs_device.h"

namespace bs {

constexpr int kTile = 128;
constexpr int kThreads = 256;

struct Raw {
    uint4 v[8];  // v[i]: row 8*tr + i, columns 8*tc .. +7 (bf16)
};

struct TileRegs {
    float f[8][8];  // f[i][j]: row 8*tr + i, column 8*tc + j of the tile
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Raw buffer over [base, base + bytes): loads past the end read zero and
// stores past the end are dropped, which handles ragged tiles without
// per-lane bounds checks; the tile origin lives in the (scalar) descriptor
// and lanes keep 32-bit offsets.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
    const int32_t n = bytes > 0x7fffffff ? 0x7fffffff : (bytes < 0 ? 0 : (int32_t)bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, 0x00020000);
}

// Rows [r0, r0 + 128) of a tile whose first column is c0; rows >= R read as 0.
__device__ __forceinline__ void load_raw(const uint16_t* __restrict__ x, int64_t ld_x, int64_t r0, int64_t c0,
                                         int64_t R, int voff, Raw& raw) {
    const int64_t rows = (R - r0) < kTile ? (R - r0) : kTile;
    const __amdgpu_buffer_rsrc_t rx = rsrc(x + r0 * ld_x + c0, rows * ld_x * 2);
    const int row_bytes = (int)(ld_x * 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, voff, i * row_bytes, 0));
        raw.v[i] = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

__device__ __forceinline__ void unpack_tile(const Raw& raw, TileRegs& t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack8(raw.v[i], t.f[i]);
}

// Transposed store of an 8x8 block of codes per thread through LDS.
// codes[j] holds the 8 codes of column 8*tc + j for rows 8*tr .. 8*tr + 7.
// LDS tile: row c (a column of the source) is 128 bytes = 16 chunks of 8
// bytes; chunk tr is stored at physical chunk tr ^ tc, which spreads the 16
// lanes of a DPP row over all banks.  `out` points at output row 0, column 0
// of the tile; 8 lanes write each 128-byte output row.
__device__ __forceinline__ void store_transposed(uint8_t* lds, const uint2* codes, int tr, int tc,
                                                 uint8_t* __restrict__ out, int64_t ld_out) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = 8 * tc + j;
        *reinterpret_cast<uint2*>(lds + c * kTile + ((tr ^ tc) * 8)) = codes[j];
    }
    __syncthreads();
    const int t = threadIdx.x;
    const __amdgpu_buffer_rsrc_t ro = rsrc(out, (kTile - 1) * ld_out + kTile);
    const int voff = (t >> 3) * (int)ld_out + 16 * (t & 7);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int c = p * 32 + (t >> 3);
        const int k = t & 7;          // 16-byte chunk of the output row
        const int sw = (c >> 3) & 15;  // swizzle of LDS row c
        const int phys = (2 * k) ^ sw;  // physical 8-byte chunk of logical chunk 2k
        uint4 v = *reinterpret_cast<const uint4*>(lds + c * kTile + (phys & ~1) * 8);
        if (sw & 1) {  // the pair is stored swapped
            v = make_uint4(v.z, v.w, v.x, v.y);
        }
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{v.x, v.y, v.z, v.w}, ro, voff, p * 32 * (int)ld_out, 0);
    }
}

__device__ __forceinline__ void col_codes(const TileRegs& tile, const Scale* sc, uint2* codes) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        codes[j].x = encode4(div_by_scale(tile.f[0][j], sc[j]), div_by_scale(tile.f[1][j], sc[j]),
                             div_by_scale(tile.f[2][j], sc[j]), div_by_scale(tile.f[3][j], sc[j]));
        codes[j].y = encode4(div_by_scale(tile.f[4][j], sc[j]), div_by_scale(tile.f[5][j], sc[j]),
                             div_by_scale(tile.f[6][j], sc[j]), div_by_scale(tile.f[7][j], sc[j]));
    }
}

// ---- the FFN's gated activation h = silu(a) * b and its derivative ----
// The value quantized is the float64 formula rounded once to bf16 (nearest
// even).  Each kernel evaluates it in fp32 (relative error below 2^-20 where
// no intermediate leaves the normal range) and takes that value's bf16
// rounding unless it lies within the error bound of a rounding tie, where
// (rarely) the float64 formula is evaluated instead.

// Distance of r from the nearest bf16 rounding tie, in fp32 units in the last
// place (the low 16 bits of r against the half step 0x8000).
__device__ __forceinline__ float tie_distance(float r) {
    // in float: the low half-word and its distance to 0x8000 are small
    // integers, exact in fp32 (4 instructions with the caller's - 16, against
    // 7 for the integer form)
    return fabsf((float)(__float_as_uint(r) & 0xFFFFu) - 32768.0f);
}

// float64 -> bf16 (as float), nearest even, one rounding: the fp64 -> fp32
// step rounds to odd (truncate, set the last bit if inexact), which keeps 16
// more bits than bf16, so the final fp32 -> bf16 rounding is the correct one.
__device__ __forceinline__ float bf16_from_double(double d) {
    float f = (float)d;
    if ((double)f != d) {
        uint32_t u = __float_as_uint(f);
        if (fabs((double)f) > fabs(d)) u -= 1u;  // step toward zero (inf -> FLT_MAX)
        f = __uint_as_float(u | 1u);
    }
    return (float)(__bf16)f;
}

constexpr float kTieWindow = 16.0f;   // fp32 ulps; the fp32 paths err by < 8

// tie_distance(r) > kTieWindow in two 16-bit integer instructions: the low
// half-word of r shifted so that the window [0x8000 - 16, 0x8000 + 16] maps
// to [0, 32].
__device__ __forceinline__ bool off_tie(float r) {
    return (uint16_t)(__float_as_uint(r) - (0x8000u - 16u)) > 32u;
}
constexpr float kMinNormal = 1.17549435e-38f;  // 2^-126

// The float64 evaluations, for the few elements in a thousand the fp32 paths
// leave undecided; each kernel calls them from one per-lane loop, outside its
// unrolled fp32 code.
__device__ __forceinline__ float swiglu_bf16_f64(float a, float b) {
    const double ad = a;
    return bf16_from_double(ad / (1.0 + exp(-ad)) * (double)b);
}

// da and db in float64 for the elements the fp32 path leaves undecided.
__device__ __forceinline__ float2 swiglu_grad_bf16_f64(float a, float b, float dh) {
    const double ad = a, bd = b, dd = dh;
    const double sd = 1.0 / (1.0 + exp(-ad));
    const double snd = 1.0 / (1.0 + exp(ad));
    return make_float2(bf16_from_double(dd * bd * sd * (1.0 + ad * snd)), bf16_from_double(dd * (ad * sd)));
}

// Undecided elements come out as +inf (bf16 0x7F80), which marks them for the
// float64 pass (the fp32 paths never return a true infinity: it is undecided).
constexpr uint32_t kRedoBits = 0x7F80u;

// exp(-a) in fp32 from the hardware base-2 exponential: -a log2(e) is
// formed as a rounded head ph plus its tail pl (the product's rounding error,
// exact by fma, and the part of log2(e) below fp32), and 2^(ph + pl) is taken
// as 2^ph (1 + pl ln 2).  On every bf16 value a with a normal result this is
// within 1.12 fp32 ulps of exp(-a) (the library expf: 0.76 ulps), at 6
// instructions instead of 13; results below the normal range come out as 0,
// where 1 + exp(-a) is 1 anyway.
constexpr float kLog2e = 1.44269502162933349609375f;  // log2(e) rounded to fp32
constexpr float kLog2eTail = 1.925963e-08f;           // log2(e) - kLog2e
constexpr float kLn2 = 0.693147180559945309f;
__device__ __forceinline__ float exp_neg(float a) {
    const float ph = -a * kLog2e;
    const float pl = __builtin_fmaf(-a, kLog2eTail, __builtin_fmaf(-a, kLog2e, -ph));
    const float e = __builtin_amdgcn_exp2f(ph);
    return __builtin_fmaf(e, pl * kLn2, e);
}

// h = silu(a) * b in fp32, to be rounded once to bf16 (nearest even) by the
// caller's packing; +inf (to be redone in float64) where a <= -69 (exp(-a)
// near fp32 overflow), silu(a) is subnormal,
// the product is not finite, or it lies near a rounding tie.  The quotient is
// a times the hardware reciprocal of 1 + exp(-a) (1 ulp; 1 + exp(-a) >= 1 is
// never subnormal); with exp_neg's 1.12 ulps the fp32 value errs by < 8 ulps,
// half the tie window.
__device__ __forceinline__ float swiglu_fast(float a, float b) {
    const float silu = a * __builtin_amdgcn_rcpf(1.0f + exp_neg(a));
    const float r = silu * b;
    const bool normal = silu == 0.0f || fabsf(silu) >= kMinNormal;
    const bool ok = a > -69.0f && normal && __builtin_isfinite(r) && off_tie(r);
    return ok ? r : __builtin_inff();
}

// da = dh * b * silu'(a) and db = dh * silu(a), silu'(a) = s (1 + a (1 - s)),
// s = 1 / (1 + exp(-a)), in fp32, each to be rounded once to bf16 by the
// caller's packing; da = +inf where
// either rounding is not certain to be the float64 formula's (a <= -69,
// an intermediate outside the normal range, or a value near a tie).  One
// exponential serves both sigmoids: 1 - s = exp(-a) s (within 2.3 ulps of
// 1 / (1 + exp(a)) on every bf16 a, as s is of its value).  Near
// silu'(a) = 0 the sum t = 1 + a (1 - s) cancels, so da's window adds
// 8 |a (1 - s)| / |t| ulps (infinite at t = 0), written without a division.
// The reciprocal is the hardware's (1 ulp; its argument is >= 1, never
// subnormal), inside both windows' margins.
__device__ __forceinline__ void swiglu_grad_fast(float a, float b, float dh, float& da, float& db) {
    const float e = exp_neg(a);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    const float sn = e * s;
    const float t = __builtin_fmaf(a, sn, 1.0f);
    const float p1 = dh * b, p2 = p1 * s;
    const float rda = p2 * t;
    const float silu = a * s;
    const float rdb = dh * silu;
    // bitwise & of the conditions: all are cheap to evaluate, and
    // short-circuit && would make the compiler branch per element
    const bool ok_a = __builtin_isfinite(rda) &
                      ((p1 == 0.0f) | ((fabsf(p1) >= kMinNormal) & (fabsf(p2) >= kMinNormal))) &
                      ((tie_distance(rda) - kTieWindow) * fabsf(t) > 8.0f * fabsf(a * sn));
    const bool ok_b = __builtin_isfinite(rdb) & ((silu == 0.0f) | (fabsf(silu) >= kMinNormal)) & off_tie(rdb);
    const bool ok = (a > -69.0f) & ok_a & ok_b;
    da = ok ? rda : __builtin_inff();
    db = rdb;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) | ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16);
}

// Word k (0..31, static) of a thread's packed 8x8 block: row k / 4,
// columns 2 (k % 4) and 2 (k % 4) + 1.
__device__ __forceinline__ uint32_t raw_word(const Raw& r, int k) {
    const uint4 v = r.v[k >> 2];
    return (k & 3) == 0 ? v.x : (k & 3) == 1 ? v.y : (k & 3) == 2 ? v.z : v.w;
}

// Replaces element e (per lane: row e / 8, column e % 8) of a packed block by
// a bf16-exact value (rare path).  Branch-free blends: every word is rewritten
// with a mask that is zero except at the target half-word, so the block stays
// in registers (per-word conditional stores can be turned into an indexed
// store, which puts the block in private memory).
__device__ __forceinline__ void raw_set(Raw& r, int e, float v) {
    const uint32_t w = (uint32_t)e >> 1;
    const uint32_t h16 = __float_as_uint(v) >> 16;
    const uint32_t field = (e & 1) ? 0xFFFF0000u : 0x0000FFFFu;
    const uint32_t put = (e & 1) ? (h16 << 16) : h16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t mx = (4u * i + 0u == w) ? field : 0u, my = (4u * i + 1u == w) ? field : 0u;
        const uint32_t mz = (4u * i + 2u == w) ? field : 0u, mw = (4u * i + 3u == w) ? field : 0u;
        r.v[i].x = (r.v[i].x & ~mx) | (put & mx);
        r.v[i].y = (r.v[i].y & ~my) | (put & my);
        r.v[i].z = (r.v[i].z & ~mz) | (put & mz);
        r.v[i].w = (r.v[i].w & ~mw) | (put & mw);
    }
}

// Re-evaluates, in float64, the elements of a thread's packed block that the
// fp32 path marked (+inf); fn(e) does element e.  The marks are found with
// integer arithmetic only (per-element compares would keep 64 lane masks
// alive), and the loop runs per lane: a wave spends one pass per marked
// element of its busiest lane (usually none or one per tile).
template <typename F>
__device__ __forceinline__ void fixup_block(const Raw& marked, F&& fn) {
    uint32_t m[2] = {0u, 0u};  // elements 0..31, 32..63
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const uint32_t w = raw_word(marked, k);
        const uint32_t lo = ((w & 0xFFFFu) ^ kRedoBits) - 1u, hi = ((w >> 16) ^ kRedoBits) - 1u;
        m[k >> 4] |= ((lo >> 31) << ((2 * k) & 31)) | ((hi >> 31) << ((2 * k + 1) & 31));
    }
    for (int h = 0; h < 2; ++h) {
        uint32_t mask = m[h];
        while (mask != 0) {
            const int e = 32 * h + __builtin_ctz(mask);
            mask &= mask - 1;
            fn(e);
        }
    }
}

// 1x128 row blocks of one tile: codes to q (the tile's first element; rows
// past `rows` are dropped), scales to s (the tile's entries of one K-major
// scale row).
__device__ __forceinline__ void quant_tile_rows(const TileRegs& tl, int64_t rows, uint8_t* q, int64_t ld_q,
                                                float* s, int tr, int tc) {
    const __amdgpu_buffer_rsrc_t rq = rsrc(q, rows * ld_q);
    const int voff_q = (8 * tr) * (int)ld_q + 8 * tc;
    float my_scale = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(tl.f[i][j]));
        const uint32_t amax_bits = row16_max(__float_as_uint(m));
        const Scale sc = block_scale(__uint_as_float(amax_bits));
        const uint2 qv = quant8(tl.f[i], sc);
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{qv.x, qv.y}, rq, voff_q, i * (int)ld_q, 0);
        if ((tc & 7) == i) my_scale = sc.s;
    }
    // lanes tc < 8 store the scale of row 8*tr + tc: 32 consecutive rows per wave
    const __amdgpu_buffer_rsrc_t rs = rsrc(s, rows * 4);
    if (tc < 8) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(my_scale), rs, (8 * tr + tc) * 4, 0, 0);
}

// 1x128 column blocks (the tile's 128 rows) of one tile: codes written
// transposed to qt (row c0 of q^T, column r0), scales to s (128 consecutive
// entries of one K-major scale row).  colmax and tr_lds are this call's LDS
// buffers (alternate between consecutive calls); it holds barriers, so every
// thread of the workgroup calls it.
__device__ __forceinline__ void quant_tile_cols(const TileRegs& tl, uint8_t* qt, int64_t ld_qt, float* s,
                                                float (*colmax)[kTile], uint8_t* tr_lds, int tr, int tc, int wave) {
    float cm[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(tl.f[i][j]));
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        cm[j] = m;
    }
    if ((threadIdx.x & 63) < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) colmax[wave][8 * tc + j] = cm[j];
    }
    __syncthreads();
    Scale sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = 8 * tc + j;
        const float m = fmaxf(fmaxf(colmax[0][c], colmax[1][c]), fmaxf(colmax[2][c], colmax[3][c]));
        sc[j] = block_scale(m);
    }
    uint2 codes[8];
    col_codes(tl, sc, codes);
    if (threadIdx.x < 16) {
        const __amdgpu_buffer_rsrc_t rs = rsrc(s, kTile * 4);
        __builtin_amdgcn_raw_buffer_store_b128(
            u32x4{__float_as_uint(sc[0].s), __float_as_uint(sc[1].s), __float_as_uint(sc[2].s),
                  __float_as_uint(sc[3].s)}, rs, 32 * tc, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(
            u32x4{__float_as_uint(sc[4].s), __float_as_uint(sc[5].s), __float_as_uint(sc[6].s),
                  __float_as_uint(sc[7].s)}, rs, 32 * tc + 16, 0, 0);
    }
    store_transposed(tr_lds, codes, tr, tc, qt, ld_qt);
}

// bf16 values of a tile's rows (already bf16-exact floats) -> packed rows.
__device__ __forceinline__ void pack_tile(const TileRegs& tl, Raw& raw) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        raw.v[i] = make_uint4(pack_bf16(tl.f[i][0], tl.f[i][1]), pack_bf16(tl.f[i][2], tl.f[i][3]),
                              pack_bf16(tl.f[i][4], tl.f[i][5]), pack_bf16(tl.f[i][6], tl.f[i][7]));
}

// Packed rows of a tile to out (the tile's first element; rows past `rows`
// are dropped).
__device__ __forceinline__ void store_raw(const Raw& raw, uint16_t* out, int64_t ld_out, int64_t rows, int tr,
                                          int tc) {
    const __amdgpu_buffer_rsrc_t ro = rsrc(out, rows * ld_out * 2);
    const int voff = (8 * tr) * (int)(ld_out * 2) + 16 * tc;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{raw.v[i].x, raw.v[i].y, raw.v[i].z, raw.v[i].w}, ro, voff,
                                               i * (int)(ld_out * 2), 0);
}

}  // namespace bs
