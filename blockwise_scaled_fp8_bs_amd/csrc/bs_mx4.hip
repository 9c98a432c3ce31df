// MXFP4 quantizer of weights: 32 consecutive values of a row share a scale
// 2^e, e = floor(log2 amax) - 2 (the exponent of 6, e2m1's largest), clamped
// to [-127, 127]; the byte e + 127 of a normal amax is its exponent field
// minus 2, so no logarithm is taken.  Elements are e2m1(x / 2^e), nearest
// even, saturating: v_cvt_scalef32_pk_fp4_bf16 does exactly this from the bf16
// pair and the byte in an exponent field (checked on the device for every
// bf16 pattern and every byte, subnormals among them).
//
// Bound by HBM: 2 bytes in, 0.53 out (2.53 with the values): 65536 x 5120 with
// the values 276 us, 5.5 TB/s.
#include "bs_few.h"
#include "bs_tile.h"

namespace bs {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kQRows = 32, kQCols = 256;  // a workgroup's tile: 512-byte row segments in, 128-byte ones of codes out

}  // namespace

// Thread t: columns 8 (t % 32) .. +7 of the rows t / 32 + 8 i; a block of 32
// columns is a lane quad's.
__global__ __launch_bounds__(256) void mx4_quant_kernel(Mx4QuantArgs a) {
    __shared__ uint8_t s_byte[kQCols / 32][kQRows];
    const int t = threadIdx.x;
    // Neighbouring tiles share cache lines where rows are no whole number of them, and run on one XCD (37641 x 2720: 91
    // us, 107 in the order of the workgroups).
    const uint32_t tile = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3), cols_of = (uint32_t)a.col_tiles;
    const int64_t r0 = (int64_t)(tile / cols_of) * kQRows, c0 = (int64_t)(tile % cols_of) * kQCols;
    if (r0 >= a.R) return;
    const int rows = (int)(a.R - r0 < kQRows ? a.R - r0 : kQRows);
    const int cols = (int)(a.C - c0 < kQCols ? a.C - c0 : kQCols);
    const int c = 8 * (t & 31), r = t >> 5;
    const bool in = c < cols;  // (a lane quad's columns are in or out together)
    u32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = u32x4{0, 0, 0, 0};
        if (in && r + 8 * i < rows)
            v[i] = *reinterpret_cast<const u32x4*>(a.x + (r0 + r + 8 * i) * a.ld_x + c0 + c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, max((v[i][j] & 0x7fffu) << 16, v[i][j] & 0x7fff0000u));
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
        const uint32_t ex = m >> 23, byte = ex > 2u ? ex - 2u : 0u;
        const float scale = __uint_as_float(byte << 23);
        const uint32_t p[4] = {v[i][0], v[i][1], v[i][2], v[i][3]};
        uint32_t q = 0;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p[0]), scale, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p[1]), scale, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p[2]), scale, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p[3]), scale, 3);
        if ((t & 3) == 0) s_byte[(t & 31) >> 2][r + 8 * i] = (uint8_t)byte;
        if (in && r + 8 * i < rows) {
            const int64_t row = r0 + r + 8 * i;
            *reinterpret_cast<uint32_t*>(a.q + row * a.ld_q + (c0 + c) / 2) = q;
            if (a.y) {
                u32x4 y;
                y[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0));
                y[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1));
                y[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2));
                y[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3));
                *reinterpret_cast<u32x4*>(a.y + row * a.ld_y + c0 + c) = y;
            }
        }
    }
    __syncthreads();
    // one byte a thread: 32 consecutive rows of a block
    const int b = t >> 5, row = t & 31;
    if (32 * b < cols && row < rows) a.s[(c0 / 32 + b) * a.ld_s + r0 + row] = s_byte[b][row];
}

hipError_t launch_mx4_quant(const Mx4QuantArgs& args, hipStream_t stream) {
    Mx4QuantArgs a = args;
    a.col_tiles = (a.C + kQCols - 1) / kQCols;
    const int64_t tiles = (a.R + kQRows - 1) / kQRows * a.col_tiles;
    hipLaunchKernelGGL(mx4_quant_kernel, dim3((unsigned)((tiles + 7) & ~7)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace bs
