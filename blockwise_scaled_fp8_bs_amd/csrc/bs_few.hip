// Few tokens through quantized weights: the product of few rows, and the gated
// experts of an MoE layer with their weighted sum.
//
// Every weight is read once and meets few tokens, so that the bytes of the
// weights bound the time.  The weights are the first operand of
// v_mfma_f32_16x16x32_bf16 (16 of their rows a tile), the tokens the second
// (16 a tile): a lane's 16 bytes of codes go from global memory into its
// registers, are converted to bf16 there (exact: e4m3 and e2m1 fit, and MX
// scales are powers of two that the conversion applies) and multiply at once.
// The waves of a workgroup take turns along the contraction, 128 values at a
// time (a unit), and add their sums up at the end in a fixed order.  Tokens
// and rows that are not there are read as zeros by the buffers' bounds.
//
// Tokens stay in bf16: quantizing them would save nothing where the weights
// are the traffic.  Sums are in fp32.
#include "bs_few.h"
#include "bs_tile.h"

namespace bs {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kUnit = 128;            // values along the contraction that a wave takes at a time
constexpr int kOut = 0x70000000;      // an offset past every buffer: reads zero

// Weights of NT tiles of 16 rows and tokens of TT tiles of 16, for one unit.
// e4m3: lane (r, g) = (l % 16, l / 16) holds row r's values 16 g .. +15 of each
// half of the unit; e2m1: its values 32 g .. +31.
template <int KIND, int NT, int TT>
struct Frag {
    static constexpr int kLoads = KIND == kFewMx4 ? 1 : 2;
    u32x4 a[NT][kLoads];
    uint32_t s[NT][kLoads];  // scale bytes (MX)
    float sc[NT];            // the 128x128 block's scale
    u32x4 x[TT][4];
};

// 16 rows of weights: the codes and scales that a wave reads of them.
struct Rows {
    const uint8_t* q;  // first row
    const void* s;     // its scales
    int rows;          // at most 16
};

template <int KIND>
__device__ __forceinline__ Rows tile_rows(const FewWeight& w, int64_t e, int64_t row0, int64_t N) {
    Rows t;
    t.q = w.q + e * w.stride_q + row0 * w.ld_q;
    if (KIND == kFewE4m3)
        t.s = static_cast<const float*>(w.s) + e * w.stride_s + row0 / 128;
    else
        t.s = static_cast<const uint8_t*>(w.s) + e * w.stride_s + row0;
    t.rows = (int)(N - row0 < 16 ? N - row0 : 16);
    return t;
}

template <int KIND>
__device__ __forceinline__ void load_rows(u32x4* a, uint32_t* s, float& sc, const Rows& t, int64_t ld_q, int64_t ld_s,
                                          int K, int u, int r, int g) {
    const int row_bytes = KIND == kFewMx4 ? K / 2 : K;
    const __amdgpu_buffer_rsrc_t rq = rsrc(t.q, t.rows > 0 ? (t.rows - 1) * ld_q + row_bytes : 0);
    const int row = r * (int)ld_q;
    if (KIND == kFewMx4) {
        const int k = u * kUnit + 32 * g;
        a[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rq, k < K ? row + k / 2 : kOut, 0, 0));
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = u * kUnit + 64 * h + 16 * g;
            a[h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rq, k < K ? row + k : kOut, 0, 0));
        }
    }
    if (KIND == kFewE4m3) {
        const int kb = u < K / kUnit ? u : 0;
        const float v = static_cast<const float*>(t.s)[kb * ld_s];
        sc = u < K / kUnit ? v : 0.f;
    } else {
        // the unit's four rows of scale bytes
        const int64_t left = (K / 32 - 4 * (int64_t)u - 1) * ld_s + t.rows;
        const __amdgpu_buffer_rsrc_t rs = rsrc(static_cast<const uint8_t*>(t.s) + 4 * u * ld_s, t.rows > 0 ? left : 0);
        if (KIND == kFewMx4) {
            s[0] = __builtin_amdgcn_raw_buffer_load_b8(rs, g * (int)ld_s + r, 0, 0);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) s[h] = __builtin_amdgcn_raw_buffer_load_b8(rs, (2 * h + g / 2) * (int)ld_s + r, 0, 0);
        }
    }
}

// The unit's values of a token's row, whose bytes start at `row` (kOut: none).
template <int KIND>
__device__ __forceinline__ void load_token(u32x4* x, const __amdgpu_buffer_rsrc_t rx, int row, int K, int u, int g) {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        const int k = u * kUnit + (KIND == kFewMx4 ? 32 * g + 8 * f : 64 * (f / 2) + 16 * g + 8 * (f % 2));
        x[f] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, k < K ? row + 2 * k : kOut, 0, 0));
    }
}

// Eight weights in bf16: the f-th quarter of a lane's codes.
template <int KIND>
__device__ __forceinline__ bf16x8 weights(const u32x4* a, const uint32_t* s, int f) {
    union {
        bf16x2 p[4];
        bf16x8 v;
    } w;
    if (KIND == kFewMx4) {
        const float scale = __uint_as_float(s[0] << 23);
        const uint32_t c = a[0][f];
        w.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
        w.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
        w.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
        w.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
    } else {
        const float scale = KIND == kFewMx8 ? __uint_as_float(s[f / 2] << 23) : 1.f;
        const uint32_t c0 = a[f / 2][2 * (f % 2)], c1 = a[f / 2][2 * (f % 2) + 1];
        w.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, scale, false);
        w.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, scale, true);
        w.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, scale, false);
        w.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, scale, true);
    }
    return w.v;
}

template <int KIND, int NT, int TT>
__device__ __forceinline__ void multiply(const Frag<KIND, NT, TT>& f, f32x4 (&acc)[NT][TT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        f32x4 p[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) p[t] = KIND == kFewE4m3 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[n][t];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x8 w = weights<KIND>(f.a[n], f.s[n], j);
#pragma unroll
            for (int t = 0; t < TT; ++t)
                p[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, f.x[t][j]), p[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[n][t][i] = KIND == kFewE4m3 ? __builtin_fmaf(p[t][i], f.sc[n], acc[n][t][i]) : p[t][i];
    }
}

// Units of one wave, DEPTH of them in flight: load(frag, i) reads the wave's
// i-th unit, zeros past its `units`.
template <int KIND, int NT, int TT, int DEPTH, class Load>
__device__ __forceinline__ void stream_units(int units, f32x4 (&acc)[NT][TT], Load load) {
    Frag<KIND, NT, TT> f[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(f[d], d);
    for (int i = 0; i < units; i += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            multiply<KIND, NT, TT>(f[d], acc);
            load(f[d], i + DEPTH + d);
        }
    }
}

template <int NT, int TT>
__device__ __forceinline__ void zero(f32x4 (&acc)[NT][TT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Each wave's sums into LDS: red[wave][tile][lane], tile = n * TT + t.
template <int NT, int TT>
__device__ __forceinline__ void put_sums(f32x4* red, int wave, int lane, const f32x4 (&acc)[NT][TT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < TT; ++t) red[(wave * NT * TT + n * TT + t) * 64 + lane] = acc[n][t];
}

// The waves' sums of one lane's place in a tile, in the order of the waves.
template <int W, int TILES>
__device__ __forceinline__ f32x4 sum_waves(const f32x4* red, int tile, int lane) {
    f32x4 v = red[tile * 64 + lane];
#pragma unroll
    for (int w = 1; w < W; ++w) {
        const f32x4 o = red[(w * TILES + tile) * 64 + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += o[i];
    }
    return v;
}

__device__ __forceinline__ uint32_t bf16_bits(float f) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}

// Four consecutive columns of a row of the output, on the residual.
__device__ __forceinline__ void store4(f32x4 v, const uint16_t* residual, void* out, bool f32, bool vec, int cols) {
    if (vec) {
        if (residual) {
            const uint2 q = *reinterpret_cast<const uint2*>(residual);
            v = f32x4{bf16_lo(q.x) + v[0], bf16_hi(q.x) + v[1], bf16_lo(q.y) + v[2], bf16_hi(q.y) + v[3]};
        }
        if (f32)
            *reinterpret_cast<f32x4*>(out) = v;
        else
            *reinterpret_cast<uint2*>(out) = make_uint2(bf16_bits(v[0]) | bf16_bits(v[1]) << 16, bf16_bits(v[2]) | bf16_bits(v[3]) << 16);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= cols) break;
        const float o = residual ? bf16_lo(residual[i]) + v[i] : v[i];
        if (f32)
            static_cast<float*>(out)[i] = o;
        else
            static_cast<uint16_t*>(out)[i] = (uint16_t)bf16_bits(o);
    }
}

// Neighbouring tiles share the cache lines of MX scale bytes (128 rows a line)
// and run on one XCD: workgroup b of `padded` (a multiple of 8) takes this one.
__device__ __forceinline__ int xcd_tile(int b, int padded) { return (b & 7) * (padded >> 3) + (b >> 3); }

// ---------------------------------------------------------------------------
// out = residual + x W^T
// ---------------------------------------------------------------------------

template <int KIND, int NT, int TT, int W, int DEPTH>
__global__ __launch_bounds__(64 * W) void few_mm_kernel(FewMmArgs a) {
    __shared__ f32x4 red[W * NT * TT * 64];
    const int tile = xcd_tile(blockIdx.x, gridDim.x);
    if (tile >= a.tiles) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.y * kFewChunk, row0 = (int64_t)tile * (16 * NT);
    const int T = (int)(a.T - t0 < 16 * TT ? a.T - t0 : 16 * TT), K = (int)a.K;
    const __amdgpu_buffer_rsrc_t rx = rsrc(a.x + t0 * a.ld_x, ((T - 1) * a.ld_x + K) * 2);
    Rows rows[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) rows[n] = tile_rows<KIND>(a.w, 0, row0 + 16 * n, a.N);
    f32x4 acc[NT][TT];
    zero(acc);
    const int units = (K + kUnit - 1) / kUnit;
    stream_units<KIND, NT, TT, DEPTH>((units - wave + W - 1) / W, acc, [&](Frag<KIND, NT, TT>& f, int i) {
        const int u = wave + i * W;
#pragma unroll
        for (int n = 0; n < NT; ++n) load_rows<KIND>(f.a[n], f.s[n], f.sc[n], rows[n], a.w.ld_q, a.w.ld_s, K, u, r, g);
#pragma unroll
        for (int t = 0; t < TT; ++t)
            load_token<KIND>(f.x[t], rx, 16 * t + r < T ? (16 * t + r) * (int)a.ld_x * 2 : kOut, K, u, g);
    });
    put_sums(red, wave, lane, acc);
    __syncthreads();
    for (int i = threadIdx.x; i < NT * TT * 64; i += 64 * W) {
        const int id = i >> 6, l = i & 63;
        const int64_t n = row0 + 16 * (id / TT) + 4 * (l >> 4);
        const int t = 16 * (id % TT) + (l & 15);
        if (t >= T || n >= a.N) continue;
        const f32x4 v = sum_waves<W, NT * TT>(red, id, l);
        const int64_t at = (t0 + t) * a.ld_out + n;
        store4(v, a.residual ? a.residual + (t0 + t) * a.ld_res + n : nullptr,
               a.f32 ? (void*)(static_cast<float*>(a.out) + at) : (void*)(static_cast<uint16_t*>(a.out) + at), a.f32, a.vec,
               (int)(a.N - n < 4 ? a.N - n : 4));
    }
}

// ---------------------------------------------------------------------------
// gated experts: h of the routed slots, then their weighted sum
// ---------------------------------------------------------------------------

constexpr int kMaxSlots = (int)kFewChunk * 32;  // of a chunk

// The chunk's choices into LDS (-1: none) and the experts among them as bits.
template <int THREADS>
__device__ __forceinline__ void load_choices(const MoeFewArgs& a, int64_t t0, int slots, int32_t* idx, uint32_t* bits) {
    const int tid = threadIdx.x;
    if (tid < 32) bits[tid] = 0;
    __syncthreads();
    for (int i = tid; i < slots; i += THREADS) {
        int32_t e = a.idx ? a.idx[t0 * a.k + i] : 0;
        if ((uint32_t)e >= (uint32_t)a.E) e = -1;
        idx[i] = e;
        if (e >= 0) atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
}

// Sum over the lanes up to this one (32 lanes with values).
__device__ __forceinline__ int prefix_sum(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Workgroup: 16 columns of h of the rank-th expert that a token of the chunk
// chose, for all its tokens.  A token that names an expert twice counts once,
// with the sum of its weights.
template <int KIND, int TT, int W, int DEPTH>
__global__ __launch_bounds__(64 * W) void moe_few_up_kernel(MoeFewArgs a) {
    __shared__ f32x4 red[W * 2 * TT * 64];
    __shared__ int32_t s_idx[kMaxSlots];
    __shared__ uint32_t s_bits[32];
    __shared__ int32_t s_slot[kFewChunk];
    __shared__ float s_w[kFewChunk];
    const int padded = (int)((a.tiles + 7) & ~7);
    const int rank = blockIdx.x / padded, tile = xcd_tile(blockIdx.x % padded, padded);
    if (tile >= a.tiles) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.y * kFewChunk;
    const int T = (int)(a.T - t0 < kFewChunk ? a.T - t0 : kFewChunk);
    load_choices<64 * W>(a, t0, T * a.k, s_idx, s_bits);

    const uint32_t word = lane < 32 ? s_bits[lane] : 0;
    const int upto = prefix_sum(__popc(word), lane);
    if (rank >= __shfl(upto, 31)) return;
    const int at = __ffsll((unsigned long long)__ballot(lane < 32 && upto > rank)) - 1;
    uint32_t left = __shfl((int)word, at);
    for (int skip = rank - (__shfl(upto, at) - __popc(left)); skip > 0; --skip) left &= left - 1;
    const int e = __builtin_amdgcn_readfirstlane(32 * at + __ffs((int)left) - 1);

    int first = -1;
    float weight = 0.f;
    if (lane < T)
        for (int j = a.k - 1; j >= 0; --j)
            if (s_idx[lane * a.k + j] == e) {
                first = j;
                weight += a.w ? a.w[(t0 + lane) * a.k + j] : 1.f;
            }
    const unsigned long long mine = __ballot(first >= 0);
    const int count = __popcll(mine);
    if (wave == 0 && first >= 0) {
        const int c = __popcll(mine & ((1ull << lane) - 1));
        s_slot[c] = lane * a.k + first;
        s_w[c] = weight;
    }
    __syncthreads();

    const int r = lane & 15, g = lane >> 4;
    const int D = (int)a.D;
    const int64_t h0 = 16 * (int64_t)tile;
    const Rows rows[2] = {tile_rows<KIND>(a.w12, e, h0, a.H), tile_rows<KIND>(a.w12, e, a.H + h0, 2 * a.H)};
    const __amdgpu_buffer_rsrc_t rx = rsrc(a.x + t0 * a.ld_x, ((T - 1) * a.ld_x + D) * 2);
    const int units = (D + kUnit - 1) / kUnit;
    for (int c0 = 0; c0 < count; c0 += 16 * TT) {
        int token[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int c = c0 + 16 * t + r;
            token[t] = c < count ? s_slot[c] / a.k * (int)a.ld_x * 2 : kOut;
        }
        f32x4 acc[2][TT];
        zero(acc);
        stream_units<KIND, 2, TT, DEPTH>((units - wave + W - 1) / W, acc, [&](Frag<KIND, 2, TT>& f, int i) {
            const int u = wave + i * W;
#pragma unroll
            for (int n = 0; n < 2; ++n)
                load_rows<KIND>(f.a[n], f.s[n], f.sc[n], rows[n], a.w12.ld_q, a.w12.ld_s, D, u, r, g);
#pragma unroll
            for (int t = 0; t < TT; ++t) load_token<KIND>(f.x[t], rx, token[t], D, u, g);
        });
        put_sums(red, wave, lane, acc);
        __syncthreads();
        for (int i = threadIdx.x; i < TT * 64; i += 64 * W) {
            const int t = i >> 6, l = i & 63, c = c0 + 16 * t + (l & 15);
            const int64_t col = h0 + 4 * (l >> 4);
            if (c >= count || col >= a.H) continue;
            const f32x4 ga = sum_waves<W, 2 * TT>(red, t, l), up = sum_waves<W, 2 * TT>(red, TT + t, l);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = bf16_bits(s_w[c] * (ga[j] / (1.f + __expf(-ga[j])) * up[j]));
            *reinterpret_cast<uint2*>(a.h + (t0 * a.k + s_slot[c]) * a.H + col) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
        }
        __syncthreads();
    }
}

// Workgroup: 16 columns of the output of every token of the chunk, summed over
// the experts in ascending order: the weights are in h already, so that the
// sums stay in the accumulators from one expert to the next.
template <int KIND, int TT, int W, int DEPTH>
__global__ __launch_bounds__(64 * W) void moe_few_down_kernel(MoeFewArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];
    f32x4* const red = reinterpret_cast<f32x4*>(s_dyn);  // after the products: the choices' table is through then
    uint8_t* const s_choice = s_dyn;                     // [rank][token]: the choice j that names the expert, 255 for none
    __shared__ int32_t s_idx[kMaxSlots];
    __shared__ uint32_t s_bits[32];
    __shared__ int32_t s_base[32];
    __shared__ uint16_t s_expert[1024];
    const int tile = xcd_tile(blockIdx.x, gridDim.x);
    if (tile >= a.tiles) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.y * kFewChunk;
    const int T = (int)(a.T - t0 < kFewChunk ? a.T - t0 : kFewChunk);
    load_choices<64 * W>(a, t0, T * a.k, s_idx, s_bits);
    const uint32_t word = lane < 32 ? s_bits[lane] : 0;
    const int upto = prefix_sum(__popc(word), lane);
    const int ranks = __builtin_amdgcn_readfirstlane(__shfl(upto, 31));
    if (wave == 0 && lane < 32) s_base[lane] = upto - __popc(word);
    for (int i = threadIdx.x; i < ranks * T; i += 64 * W) s_choice[i] = 255;
    __syncthreads();
    for (int i = threadIdx.x; i < T * a.k; i += 64 * W) {
        const int e = s_idx[i];
        if (e < 0) continue;
        const int t = i / a.k, j = i % a.k;
        bool first = true;
        for (int o = 0; o < j; ++o) first &= s_idx[t * a.k + o] != e;
        const int rank = s_base[e >> 5] + __popc(s_bits[e >> 5] & ((1u << (e & 31)) - 1));
        s_expert[rank] = (uint16_t)e;
        if (first) s_choice[rank * T + t] = (uint8_t)j;
    }
    __syncthreads();

    const int r = lane & 15, g = lane >> 4;
    const int H = (int)a.H, units = (H + kUnit - 1) / kUnit;
    const int64_t d0 = 16 * (int64_t)tile;
    const __amdgpu_buffer_rsrc_t rh = rsrc(a.h + t0 * a.k * a.H, (int64_t)T * a.k * H * 2);
    f32x4 acc[1][TT];
    zero(acc);
    int rank = 0, u = wave;  // of the next unit to load: the experts' units follow one another
    while (u >= units && rank < ranks) u -= units, ++rank;
    const int all = ranks * units;
    stream_units<KIND, 1, TT, DEPTH>((all - wave + W - 1) / W, acc, [&](Frag<KIND, 1, TT>& f, int) {
        const bool there = rank < ranks;
        const int e = there ? __builtin_amdgcn_readfirstlane(s_expert[rank]) : 0;
        Rows rows = tile_rows<KIND>(a.wo, e, d0, a.D);
        if (!there) rows.rows = 0;
        load_rows<KIND>(f.a[0], f.s[0], f.sc[0], rows, a.wo.ld_q, a.wo.ld_s, H, there ? u : units, r, g);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int tok = 16 * t + r;
            const int j = there && tok < T ? s_choice[rank * T + tok] : 255;
            load_token<KIND>(f.x[t], rh, j != 255 ? (tok * a.k + j) * H * 2 : kOut, H, u, g);
        }
        for (u += W; u >= units && rank < ranks; ++rank) u -= units;
    });
    __syncthreads();
    put_sums(red, wave, lane, acc);
    __syncthreads();
    for (int i = threadIdx.x; i < TT * 64; i += 64 * W) {
        const int t = 16 * (i >> 6) + (i & 15);
        const int64_t d = d0 + 4 * ((i & 63) >> 4);
        if (t >= T || d >= a.D) continue;
        store4(sum_waves<W, TT>(red, i >> 6, i & 63), a.residual ? a.residual + (t0 + t) * a.ld_res + d : nullptr,
               a.out + (t0 + t) * a.ld_out + d, false, a.vec, 4);
    }
}

template <int KIND, int TT>
hipError_t mm(FewMmArgs a, hipStream_t stream) {
    constexpr int NT = 1, W = 8, DEPTH = 2;
    a.tiles = (a.N + 16 * NT - 1) / (16 * NT);
    const dim3 grid((unsigned)((a.tiles + 7) & ~7), (unsigned)((a.T + kFewChunk - 1) / kFewChunk));
    hipLaunchKernelGGL((few_mm_kernel<KIND, NT, TT, W, DEPTH>), grid, dim3(64 * W), 0, stream, a);
    return hipGetLastError();
}

template <int KIND, int TT>
hipError_t moe(MoeFewArgs a, hipStream_t stream) {
    constexpr int W = 8, DEPTH = 2;
    const int64_t chunks = (a.T + kFewChunk - 1) / kFewChunk, tokens = a.T < kFewChunk ? a.T : kFewChunk;
    const int64_t ranks = tokens * a.k < a.E ? tokens * a.k : a.E;
    a.tiles = (a.H + 15) / 16;
    const int64_t padded = (a.tiles + 7) & ~7;
    hipLaunchKernelGGL((moe_few_up_kernel<KIND, TT, W, DEPTH>), dim3((unsigned)(ranks * padded), (unsigned)chunks), dim3(64 * W),
                       0, stream, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    a.tiles = (a.D + 15) / 16;
    const size_t table = (size_t)(ranks * tokens), sums = (size_t)W * TT * 64 * sizeof(f32x4);
    hipLaunchKernelGGL((moe_few_down_kernel<KIND, TT, W, DEPTH>), dim3((unsigned)((a.tiles + 7) & ~7), (unsigned)chunks),
                       dim3(64 * W), table > sums ? table : sums, stream, a);
    return hipGetLastError();
}

template <int KIND>
hipError_t mm_kind(const FewMmArgs& a, hipStream_t stream) {
    return a.T <= 16 ? mm<KIND, 1>(a, stream) : a.T <= 32 ? mm<KIND, 2>(a, stream) : mm<KIND, 4>(a, stream);
}

template <int KIND>
hipError_t moe_kind(const MoeFewArgs& a, hipStream_t stream) {
    return a.T <= 16 ? moe<KIND, 1>(a, stream) : a.T <= 32 ? moe<KIND, 2>(a, stream) : moe<KIND, 4>(a, stream);
}

}  // namespace

hipError_t launch_few_mm(const FewMmArgs& a, FewKind kind, hipStream_t stream) {
    return kind == kFewE4m3 ? mm_kind<kFewE4m3>(a, stream)
           : kind == kFewMx8 ? mm_kind<kFewMx8>(a, stream) : mm_kind<kFewMx4>(a, stream);
}

hipError_t launch_moe_few(const MoeFewArgs& a, FewKind kind, hipStream_t stream) {
    return kind == kFewE4m3 ? moe_kind<kFewE4m3>(a, stream)
           : kind == kFewMx8 ? moe_kind<kFewMx8>(a, stream) : moe_kind<kFewMx4>(a, stream);
}

}  // namespace bs
