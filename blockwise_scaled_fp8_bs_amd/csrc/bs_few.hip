// Few tokens through quantized weights: the product of few rows, and the gated
// experts of an MoE layer with their weighted sum.
//
// Every weight is read once and meets few tokens, so that the bytes of the
// weights bound the time.  The weights are the first operand of
// v_mfma_f32_16x16x32_bf16 (16 of their rows a tile), the tokens the second
// (up to 16).  A wave streams units of 128 bytes along the rows through a ring
// of its own in LDS: buffer loads that bypass the registers fetch the codes,
// scales and tokens of the units ahead (whole cache lines, where the operands'
// layout would have every lane of a load in a line of its own: loading them
// into registers ran at 1.4 to 3.6 TB/s), and no wave waits for another before
// the sums are added up at the end, in a fixed order.  Codes are converted to
// bf16 on the way to the matrix cores (exact: e4m3 and e2m1 fit, and MX scales
// are powers of two that the conversion applies).  What lies outside the
// operands is read as zeros by the buffers' bounds.
//
// Tokens stay in bf16: quantizing them would save nothing where the weights
// are the traffic.  Sums are in fp32.
#include <type_traits>

#include "bs_dma.h"
#include "bs_few.h"
#include "bs_tile.h"

namespace bs {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kOut = 0x70000000;  // an offset past every buffer: reads zero

// A unit: HB bytes along each of 16 rows of codes (128; 64 for e2m1 beside many
// tokens, whose values would fill the ring).
template <int KIND, int HB>
struct Unit {
    static constexpr int kCodes = KIND == kFewMx4 ? 2 * HB : HB;   // along the contraction
    static constexpr int kPieces = HB / 16;                        // 16-byte pieces of a row
    static constexpr int kHalves = kPieces / 4;                    // pieces of a lane
    static constexpr int kSteps = kCodes / 32;                     // matrix instructions
    static constexpr int kBlocks = KIND == kFewE4m3 ? 1 : kCodes / 32;  // scales along the contraction
    static constexpr int kTokenRow = 2 * kCodes;                   // bytes of a token
    // pieces are stored xor-ed with a key of the row, so that eight rows' same piece lies in eight different banks
    static __device__ __forceinline__ int key(int row) { return HB == 128 ? row & 7 : (row >> 1) & 3; }
};

// A stage of the ring: NT tiles of 16 rows, their scales, RX tokens.
template <int KIND, int HB, int NT, int RX>
struct Stage {
    using U = Unit<KIND, HB>;
    static constexpr int kTile = 16 * HB;
    static constexpr int kScales = 16 * U::kBlocks;
    static constexpr int kScaleAt = NT * kTile, kTokenAt = kScaleAt + NT * kScales;
    static constexpr int kBytes = kTokenAt + RX * U::kTokenRow;
    static constexpr int kSlots = U::kTokenRow / 16;             // lanes of a token
    static constexpr int kCopies = RX * kSlots > 64 ? RX * kSlots / 64 : 1;  // loads of the tokens
    static constexpr int kTileLoads = kTile / 1024;
    static constexpr int kLoads = NT * (kTileLoads + 1) + kCopies;
};

constexpr int ring_stages(int ring, int stage) { return ring / stage < 6 ? ring / stage : 6; }

// 16 rows of weights.
struct Tile16 {
    i32x4 q;           // their codes
    const uint8_t* s;  // their scales' first byte
};

// The units of a wave: weights' row pieces and tokens' pieces of its lanes.
template <int KIND, int HB, int NT, int RX>
struct Loader {
    using U = Unit<KIND, HB>;
    using S = Stage<KIND, HB, NT, RX>;
    int lane, piece;               // 16-byte piece of the row that the lane fetches, in bytes
    int row[S::kTileLoads];        // offset of its row and piece
    int token[S::kCopies];         // offset of its token and piece (kOut: none)
    int K, row_bytes;
    int64_t ld_s;                  // bytes

    __device__ __forceinline__ void rows(int lane_, int64_t ld_q, int64_t ld_s_, int K_) {
        lane = lane_;
        K = K_;
        row_bytes = KIND == kFewMx4 ? K / 2 : K;
        ld_s = KIND == kFewE4m3 ? 4 * ld_s_ : ld_s_;
        constexpr int per = 64 / U::kPieces;  // rows of a load
#pragma unroll
        for (int i = 0; i < S::kTileLoads; ++i) {
            const int r = i * per + lane / U::kPieces;
            piece = 16 * ((lane % U::kPieces) ^ U::key(r));  // (the same for every i: per is a multiple of the key's period)
            row[i] = r * (int)ld_q + piece;
        }
    }
    static __device__ __forceinline__ int token_row(int i, int lane) { return i * (64 / S::kSlots) + lane / S::kSlots; }
    static __device__ __forceinline__ int token_piece(int i, int lane) {
        return 16 * ((lane % S::kSlots) ^ (token_row(i, lane) & 7));
    }
    // offset of token c's first byte by first(c), kOut for none
    template <class First>
    __device__ __forceinline__ void tokens(First first) {
#pragma unroll
        for (int i = 0; i < S::kCopies; ++i) {
            const int at = first(token_row(i, lane));
            token[i] = at == kOut ? kOut : at + token_piece(i, lane);
        }
    }

    // S::kLoads loads, whatever is there of the unit
    __device__ __forceinline__ void load(const Tile16 (&tile)[NT], const i32x4 x, int u, uint32_t lds) const {
        const int at = u * HB;
        const bool in = at + piece < row_bytes;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < S::kTileLoads; ++i)
                dma16(tile[n].q, lds + n * S::kTile + i * 1024, in ? row[i] : kOut, at);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint8_t* const s = tile[n].s + (int64_t)u * U::kBlocks * ld_s;
            if (KIND == kFewE4m3) {
                const i32x4 rs = make_rsrc(s, u * HB < row_bytes && tile[n].q[2] > 0 ? 4 : 0);
                if (lane == 0) dma4(rs, lds + S::kScaleAt + n * S::kScales, 0, 0);
            } else {
                const int64_t left = K / 32 - (int64_t)u * U::kBlocks;
                const i32x4 rs = make_rsrc(s, tile[n].q[2] > 0 && left > 0 ? (left - 1) * ld_s + 16 : 0);
                if (lane < U::kBlocks) dma16(rs, lds + S::kScaleAt + n * S::kScales, lane * (int)ld_s, 0);
            }
        }
        const int xat = u * U::kTokenRow;
#pragma unroll
        for (int i = 0; i < S::kCopies; ++i) {
            const int off = xat + token_piece(i, lane) < 2 * K ? token[i] : kOut;
            if (RX * S::kSlots >= 64 || lane < RX * S::kSlots) dma16(x, lds + S::kTokenAt + i * 1024, off, xat);
        }
    }
};

// Eight weights in bf16: the f-th step's of a lane.
template <int KIND>
__device__ __forceinline__ bf16x8 weights(const u32x4* a, const uint32_t* s, int f) {
    union {
        bf16x2 p[4];
        bf16x8 v;
    } w;
    if (KIND == kFewMx4) {
        const float scale = __uint_as_float(s[f / 4] << 23);
        const uint32_t c = a[f / 4][f % 4];
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

// A unit in registers.  Lane (r, g) = (l % 16, l / 16) multiplies row r of the
// weights with token r: pieces g and 4 + g of the row, and the token's values
// at those places.
template <int KIND, int HB, int NT, int RX>
struct Operands {
    using U = Unit<KIND, HB>;
    using S = Stage<KIND, HB, NT, RX>;
    u32x4 a[NT][U::kHalves], x[U::kSteps];
    uint32_t s[NT][U::kHalves];
    float sc[NT];

    __device__ __forceinline__ void read(const uint8_t* stage, int r, int g) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < U::kHalves; ++h)
                a[n][h] = *reinterpret_cast<const u32x4*>(stage + n * S::kTile + r * HB + 16 * ((4 * h + g) ^ U::key(r)));
        const int t = r & (RX - 1);  // the columns past the tokens are not used
#pragma unroll
        for (int f = 0; f < U::kSteps; ++f) {
            constexpr int per = U::kSteps / U::kHalves;  // steps, and 16-byte pieces of tokens, of a piece of codes
            const int p = (4 * (f / per) + g) * per + f % per;
            x[f] = *reinterpret_cast<const u32x4*>(stage + S::kTokenAt + t * U::kTokenRow + 16 * (p ^ (t & 7)));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint8_t* const sn = stage + S::kScaleAt + n * S::kScales;
            if (KIND == kFewE4m3) {
                sc[n] = *reinterpret_cast<const float*>(sn);
            } else {
#pragma unroll
                for (int h = 0; h < U::kHalves; ++h)
                    s[n][h] = sn[16 * (KIND == kFewMx4 ? 4 * h + g : 2 * h + g / 2) + r];
            }
        }
    }

    __device__ __forceinline__ void multiply(f32x4 (&acc)[NT]) const {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f32x4 p = KIND == kFewE4m3 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[n];
#pragma unroll
            for (int f = 0; f < U::kSteps; ++f)
                p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(weights<KIND>(a[n], s[n], f), __builtin_bit_cast(bf16x8, x[f]), p, 0,
                                                            0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = KIND == kFewE4m3 ? __builtin_fmaf(p[i], sc[n], acc[n][i]) : p[i];
        }
    }
};

template <int N>
__device__ __forceinline__ void wait_loads() {  // until at most N of the wave's loads are under way
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Streams `units` units through the wave's ring: load(i, lds) starts the loads
// of the wave's i-th unit (also of those past the end, which read zeros and
// keep the count), before(i) runs ahead of its products.
template <int KIND, int HB, int NT, int RX, int RING, class Load, class Before>
__device__ __forceinline__ void stream_units(const uint8_t* ring, int units, int r, int g, f32x4 (&acc)[NT], Load load,
                                             Before before) {
    using S = Stage<KIND, HB, NT, RX>;
    constexpr int DEPTH = ring_stages(RING, S::kBytes);
    static_assert(DEPTH >= 2, "a ring of two stages at least");
    static_assert((DEPTH - 1) * S::kLoads < 64, "the counter of loads under way has six bits");
    const uint32_t base = lds_addr(ring);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(d, base + d * S::kBytes);
    for (int i0 = 0; i0 < units; i0 += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int i = i0 + d;
            if (i >= units) break;
            wait_loads<(DEPTH - 1) * S::kLoads>();
            Operands<KIND, HB, NT, RX> o;
            o.read(ring + d * S::kBytes, r, g);
            wait_lds();  // the stage may be written again
            load(i + DEPTH, base + d * S::kBytes);
            before(i);
            o.multiply(acc);
        }
    }
    wait_loads<0>();
}

template <int KIND>
__device__ __forceinline__ Tile16 tile_rows(const FewWeight& w, int64_t e, int64_t row0, int64_t N, int K) {
    const int row_bytes = KIND == kFewMx4 ? K / 2 : K;
    const int64_t rows = N - row0 < 16 ? N - row0 : 16;
    Tile16 t;
    t.q = make_rsrc(w.q + e * w.stride_q + row0 * w.ld_q, rows > 0 ? (rows - 1) * w.ld_q + row_bytes : 0);
    t.s = static_cast<const uint8_t*>(w.s) + (KIND == kFewE4m3 ? 4 * (e * w.stride_s + row0 / 128) : e * w.stride_s + row0);
    return t;
}

// Each wave's sums into LDS: red[wave][n][lane].
template <int NT>
__device__ __forceinline__ void put_sums(f32x4* red, int wave, int lane, const f32x4 (&acc)[NT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) red[(wave * NT + n) * 64 + lane] = acc[n];
}

// The waves' sums of one lane's place in a tile, in the order of the waves.
template <int W, int NT>
__device__ __forceinline__ f32x4 sum_waves(const f32x4* red, int n, int lane) {
    f32x4 v = red[n * 64 + lane];
#pragma unroll
    for (int w = 1; w < W; ++w) {
        const f32x4 o = red[(w * NT + n) * 64 + lane];
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

// Workgroup: 16 columns of up to RX rows; its waves take turns along the
// contraction.
template <int KIND, int HB, int RX, int W, int RING>
__global__ __launch_bounds__(64 * W) void few_mm_kernel(FewMmArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[W * RING];
    const int tile = xcd_tile(blockIdx.x, gridDim.x);
    if (tile >= a.tiles) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.y * RX, row0 = (int64_t)tile * 16;
    const int T = (int)(a.T - t0 < RX ? a.T - t0 : RX), K = (int)a.K;
    const i32x4 x = make_rsrc(a.x + t0 * a.ld_x, ((T - 1) * a.ld_x + K) * 2);
    const Tile16 rows[1] = {tile_rows<KIND>(a.w, 0, row0, a.N, K)};
    Loader<KIND, HB, 1, RX> loader;
    loader.rows(lane, a.w.ld_q, a.w.ld_s, K);
    loader.tokens([&](int c) { return c < T ? c * (int)a.ld_x * 2 : kOut; });
    const int units = (K + Unit<KIND, HB>::kCodes - 1) / Unit<KIND, HB>::kCodes;
    f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    stream_units<KIND, HB, 1, RX, RING>(
        s_ring + wave * RING, (units - wave + W - 1) / W, r, g, acc,
        [&](int i, uint32_t lds) { loader.load(rows, x, wave + i * W, lds); }, [](int) {});
    __syncthreads();
    f32x4* const red = reinterpret_cast<f32x4*>(s_ring);
    put_sums(red, wave, lane, acc);
    __syncthreads();
    const int64_t n = row0 + 4 * g;
    if (wave != 0 || r >= T || n >= a.N) return;
    const int64_t at = (t0 + r) * a.ld_out + n;
    store4(sum_waves<W, 1>(red, 0, lane), a.residual ? a.residual + (t0 + r) * a.ld_res + n : nullptr,
           a.f32 ? (void*)(static_cast<float*>(a.out) + at) : (void*)(static_cast<uint16_t*>(a.out) + at), a.f32, a.vec,
           (int)(a.N - n < 4 ? a.N - n : 4));
}

// ---------------------------------------------------------------------------
// gated experts: h of the routed slots, then their weighted sum
// ---------------------------------------------------------------------------

// A chunk's choices in LDS: for every expert the tokens that chose it, as bits
// (one that names it twice counts once).  h lies in the order of the experts
// and, within one, of the tokens; both kernels derive it from these bits.
struct Choices {
    u64* tokens;  // [E]
    float* w;     // [slots]
    int16_t* e;   // [slots], -1: not routed
};

__host__ __device__ inline int choices_bytes(int E, int slots) { return (8 * E + 6 * slots + 15) / 16 * 16; }

__device__ __forceinline__ Choices choices_at(uint8_t* lds, int E, int slots) {
    Choices c;
    c.tokens = reinterpret_cast<u64*>(lds);
    c.w = reinterpret_cast<float*>(lds + 8 * E);
    c.e = reinterpret_cast<int16_t*>(lds + 8 * E + 4 * slots);
    return c;
}

template <int THREADS>
__device__ __forceinline__ void load_choices(const MoeFewArgs& a, int64_t t0, int slots, const Choices& c) {
    for (int i = threadIdx.x; i < a.E; i += THREADS) c.tokens[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += THREADS) {
        const int32_t e = a.idx ? a.idx[t0 * a.k + i] : 0;
        const bool routed = (uint32_t)e < (uint32_t)a.E;
        c.e[i] = (int16_t)(routed ? e : -1);
        c.w[i] = a.w ? a.w[t0 * a.k + i] : 1.f;
        if (routed) atomicOr(&c.tokens[e], 1ull << (i / a.k));
    }
    __syncthreads();
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ u64 below(int lane) { return (1ull << lane) - 1; }

// Workgroup: 16 columns of h of the rank-th expert that a token of the chunk
// chose, for all its tokens, 16 at a time.
template <int KIND, int W, int RING>
__global__ __launch_bounds__(64 * W) void moe_few_up_kernel(MoeFewArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[W * RING];
    __shared__ uint8_t s_token[W][kFewChunk];
    const int padded = (int)((a.tiles + 7) & ~7);
    const int rank = blockIdx.x / padded, tile = xcd_tile(blockIdx.x % padded, padded);
    if (tile >= a.tiles) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.y * kFewChunk;
    const int T = (int)(a.T - t0 < kFewChunk ? a.T - t0 : kFewChunk);
    const Choices ch = choices_at(s_dyn, a.E, T * a.k);
    load_choices<64 * W>(a, t0, T * a.k, ch);

    // the expert, and the rows of h before its own
    int e = -1, start = 0;
    u64 mine = 0;
    for (int e0 = 0, seen = 0; e0 < a.E; e0 += 64) {
        const u64 m = e0 + lane < a.E ? ch.tokens[e0 + lane] : 0;
        const u64 some = __ballot(m != 0);
        const u64 hit = __ballot(m != 0 && seen + __popcll(some & below(lane)) == rank);
        const int at = hit ? __ffsll(hit) - 1 : 64;
        start += wave_sum(lane < at ? __popcll(m) : 0);
        seen += __popcll(some);
        if (hit) {
            e = e0 + at;
            mine = (u64)(uint32_t)__shfl((int)(uint32_t)m, at) | (u64)(uint32_t)__shfl((int)(m >> 32), at) << 32;
            break;
        }
    }
    e = __builtin_amdgcn_readfirstlane(e);
    if (e < 0) return;
    start = __builtin_amdgcn_readfirstlane(start);
    const int count = __builtin_amdgcn_readfirstlane(__popcll(mine));
    if (mine >> lane & 1) s_token[wave][__popcll(mine & below(lane))] = (uint8_t)lane;
    wait_lds();

    const int r = lane & 15, g = lane >> 4, D = (int)a.D;
    const int64_t h0 = 16 * (int64_t)tile;
    const Tile16 rows[2] = {tile_rows<KIND>(a.w12, e, h0, a.H, D), tile_rows<KIND>(a.w12, e, a.H + h0, 2 * a.H, D)};
    const i32x4 x = make_rsrc(a.x + t0 * a.ld_x, ((T - 1) * a.ld_x + D) * 2);
    f32x4* const red = reinterpret_cast<f32x4*>(s_ring);
    for (int c0 = 0; c0 < count; c0 += 16) {
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        auto run = [&](auto rx, auto hb) {
            constexpr int RX = decltype(rx)::value, HB = decltype(hb)::value;
            Loader<KIND, HB, 2, RX> loader;
            loader.rows(lane, a.w12.ld_q, a.w12.ld_s, D);
            loader.tokens([&](int c) { return c0 + c < count ? s_token[wave][c0 + c] * (int)a.ld_x * 2 : kOut; });
            const int units = (D + Unit<KIND, HB>::kCodes - 1) / Unit<KIND, HB>::kCodes;
            stream_units<KIND, HB, 2, RX, RING>(
                s_ring + wave * RING, (units - wave + W - 1) / W, r, g, acc,
                [&](int i, uint32_t lds) { loader.load(rows, x, wave + i * W, lds); }, [](int) {});
        };
        const int left = count - c0;
        if (left <= 1)
            run(std::integral_constant<int, 1>{}, std::integral_constant<int, 128>{});
        else if (left <= 4)
            run(std::integral_constant<int, 4>{}, std::integral_constant<int, 128>{});
        else if (left <= 8)
            run(std::integral_constant<int, 8>{}, std::integral_constant<int, 128>{});
        else
            run(std::integral_constant<int, 16>{}, std::integral_constant<int, KIND == kFewMx4 ? 64 : 128>{});
        __syncthreads();
        put_sums(red, wave, lane, acc);
        __syncthreads();
        const int c = c0 + r;
        if (wave == 0 && c < count) {
            const f32x4 ga = sum_waves<W, 2>(red, 0, lane), up = sum_waves<W, 2>(red, 1, lane);
            const int t = s_token[0][c];
            float weight = 0.f;
            for (int j = 0; j < a.k; ++j)
                if (ch.e[t * a.k + j] == e) weight += ch.w[t * a.k + j];
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = bf16_bits(weight * (ga[j] / (1.f + __expf(-ga[j])) * up[j]));
            *reinterpret_cast<uint2*>(a.h + (t0 * a.k + start + c) * a.H + h0 + 4 * g) =
                make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
        }
        __syncthreads();
    }
}

// Workgroup: 16 columns of the output of every token of the chunk.  The work
// items, 16 tokens of an expert at most, follow one another; each wave streams
// an equal share of their units and adds what an item gave to sums of its own
// for every token (the weights are in h already), added up at the end in the
// order of the waves.
template <int KIND, int W, int RING>
__global__ __launch_bounds__(64 * W) void moe_few_down_kernel(MoeFewArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[W * RING];
    const int tile = xcd_tile(blockIdx.x, gridDim.x);
    if (tile >= a.tiles) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.y * kFewChunk;
    const int T = (int)(a.T - t0 < kFewChunk ? a.T - t0 : kFewChunk), slots = T * a.k;
    const Choices ch = choices_at(s_dyn, a.E, slots);
    uint8_t* at_lds = s_dyn + choices_bytes(a.E, slots);
    f32x4* const sums = reinterpret_cast<f32x4*>(at_lds);  // [wave][token][4]
    at_lds += W * T * 64;
    uint32_t* const item = reinterpret_cast<uint32_t*>(at_lds);  // expert << 16 | rows of h before it
    uint8_t* const token = at_lds + 4 * (a.items + 1);           // [row of h]
    load_choices<64 * W>(a, t0, slots, ch);
    for (int i = lane; i < T * 4; i += 64) sums[wave * T * 4 + i] = f32x4{0.f, 0.f, 0.f, 0.f};

    // every wave finds the items; the first one writes them down
    int items = 0, start = 0, most = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const u64 m = e0 + lane < a.E ? ch.tokens[e0 + lane] : 0;
        const int n = __popcll(m), its = (n + 15) >> 4;
        int n_upto = n, i_upto = its;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int on = __shfl_up(n_upto, d), oi = __shfl_up(i_upto, d);
            if (lane >= d) n_upto += on, i_upto += oi;
        }
        if (wave == 0) {
            const int s0 = start + n_upto - n, i0 = items + i_upto - its;
            for (int j = 0; j < its; ++j) item[i0 + j] = (uint32_t)(e0 + lane) << 16 | (uint32_t)(s0 + 16 * j);
            u64 left = m;
            for (int p = 0; p < n; ++p, left &= left - 1) token[s0 + p] = (uint8_t)(__ffsll(left) - 1);
        }
        most = max(most, n);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
        items += __shfl(i_upto, 63);
        start += __shfl(n_upto, 63);
    }
    items = __builtin_amdgcn_readfirstlane(items);
    start = __builtin_amdgcn_readfirstlane(start);
    most = __builtin_amdgcn_readfirstlane(most);
    if (wave == 0 && lane == 0) item[items] = (uint32_t)start;
    __syncthreads();

    const int r = lane & 15, g = lane >> 4, H = (int)a.H;
    const int64_t d0 = 16 * (int64_t)tile;
    f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    f32x4* const own = sums + wave * T * 4;
    auto rows_of = [&](int it, int& first, int& n) {
        const uint32_t v = __builtin_amdgcn_readfirstlane(item[it]), w = __builtin_amdgcn_readfirstlane(item[it + 1]);
        first = (int)(v & 0xffff);
        n = min(16, (int)(w & 0xffff) - first);
        return (int)(v >> 16);
    };
    auto run = [&](auto rx, auto hb) {
        constexpr int RX = decltype(rx)::value, HB = decltype(hb)::value;
        const int units = (H + Unit<KIND, HB>::kCodes - 1) / Unit<KIND, HB>::kCodes;
        const int all = items * units, share = (all + W - 1) / W, u0 = min(all, wave * share), mine = min(share, all - u0);
        Loader<KIND, HB, 1, RX> loader;
        loader.rows(lane, a.wo.ld_q, a.wo.ld_s, H);
        loader.tokens([&](int c) { return c * H * 2; });  // (those past the item's are outside the buffer)
        int l_item = u0 / units, l_u = u0 % units, l_left = mine;      // of the next unit to load
        int m_item = l_item, m_u = l_u;                                // of the next one to multiply
        Tile16 rows[1];
        i32x4 h;
        auto select = [&] {
            int first = 0, n = 0;
            const bool there = l_left > 0;
            const int e = rows_of(there ? l_item : 0, first, n);
            rows[0] = tile_rows<KIND>(a.wo, there ? e : 0, d0, a.D, H);
            h = make_rsrc(a.h + (t0 * a.k + first) * a.H, (int64_t)n * H * 2);
            if (!there) rows[0].q[2] = h[2] = 0;
        };
        if (mine > 0) {
            select();
            auto put = [&](int it) {
                int first, n;
                rows_of(it, first, n);
                if (r < n) {
                    f32x4* const s = own + token[first + r] * 4 + g;
                    const f32x4 v = *s;
                    *s = f32x4{v[0] + acc[0][0], v[1] + acc[0][1], v[2] + acc[0][2], v[3] + acc[0][3]};
                }
                acc[0] = f32x4{0.f, 0.f, 0.f, 0.f};
            };
            stream_units<KIND, HB, 1, RX, RING>(
                s_ring + wave * RING, mine, r, g, acc,
                [&](int, uint32_t lds) {
                    loader.load(rows, h, l_u, lds);
                    --l_left;
                    if (++l_u == units || l_left == 0) l_u = 0, ++l_item, select();
                },
                [&](int) {
                    if (m_u == units) put(m_item), m_u = 0, ++m_item;
                    ++m_u;
                });
            put(m_item);
        }
    };
    if (most <= 1)
        run(std::integral_constant<int, 1>{}, std::integral_constant<int, 128>{});
    else if (most <= 4)
        run(std::integral_constant<int, 4>{}, std::integral_constant<int, 128>{});
    else if (most <= 8)
        run(std::integral_constant<int, 8>{}, std::integral_constant<int, 128>{});
    else
        run(std::integral_constant<int, 16>{}, std::integral_constant<int, KIND == kFewMx4 ? 64 : 128>{});
    __syncthreads();
    for (int i = threadIdx.x; i < T * 4; i += 64 * W) {
        const int t = i >> 2;
        const int64_t d = d0 + 4 * (i & 3);
        if (d >= a.D) continue;
        f32x4 v = sums[i];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            const f32x4 o = sums[w * T * 4 + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += o[j];
        }
        store4(v, a.residual ? a.residual + (t0 + t) * a.ld_res + d : nullptr, a.out + (t0 + t) * a.ld_out + d, false, a.vec, 4);
    }
}

template <int KIND, int HB, int RX, int W, int RING>
hipError_t mm(FewMmArgs a, hipStream_t stream) {
    a.tiles = (a.N + 15) / 16;
    const dim3 grid((unsigned)((a.tiles + 7) & ~7), (unsigned)((a.T + RX - 1) / RX));
    hipLaunchKernelGGL((few_mm_kernel<KIND, HB, RX, W, RING>), grid, dim3(64 * W), 0, stream, a);
    return hipGetLastError();
}

template <int KIND>
hipError_t mm_kind(const FewMmArgs& a, hipStream_t stream) {
    if (a.T <= 1) return mm<KIND, 128, 1, 8, 9728>(a, stream);
    if (a.T <= 4) return mm<KIND, 128, 4, 8, 9728>(a, stream);
    if (a.T <= 8) return mm<KIND, 128, 8, 8, 14336>(a, stream);
    return mm<KIND, KIND == kFewMx4 ? 64 : 128, 16, 8, 14336>(a, stream);
}

template <int KIND>
hipError_t moe_kind(MoeFewArgs a, hipStream_t stream) {
    constexpr int WU = 4, WD = 8;
    const int64_t chunks = (a.T + kFewChunk - 1) / kFewChunk, tokens = a.T < kFewChunk ? a.T : kFewChunk;
    const int64_t slots = tokens * a.k, ranks = slots < a.E ? slots : a.E;
    a.tiles = (a.H + 15) / 16;
    const int64_t padded = (a.tiles + 7) & ~7;
    hipLaunchKernelGGL((moe_few_up_kernel<KIND, WU, 19200>), dim3((unsigned)(ranks * padded), (unsigned)chunks), dim3(64 * WU),
                       choices_bytes(a.E, (int)slots), stream, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    a.tiles = (a.D + 15) / 16;
    a.items = (int32_t)(ranks + slots / 16);
    hipLaunchKernelGGL((moe_few_down_kernel<KIND, WD, 12800>), dim3((unsigned)((a.tiles + 7) & ~7), (unsigned)chunks),
                       dim3(64 * WD), choices_bytes(a.E, (int)slots) + WD * tokens * 64 + 4 * (a.items + 1) + slots, stream, a);
    return hipGetLastError();
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
